// hca_cache.cuh -- device helpers shared by the serving kernels (hca_cache.cu,
// hca_cache_attn.cu, hca_cache_attn_tc.cu): e4m3 conversions, the block scale
// rule, block-wide scans, and the schedule of the attention over the cache.
#pragma once

#include <cuda_fp16.h>

#include "hca_common.cuh"
#include "hca_internal.h"

namespace hca {
namespace cache {

constexpr int kMaxPos = 1 << 30;      // positions stay below this
constexpr int kMinScaleExp = -96;     // smallest block scale 2^-96 (a block of zeros)
constexpr int kTileKeys = 128;        // keys of an attention tile

// Launches a kernel that is set up while the one in front of it on the stream
// still runs, and calls tc::pdl_wait before it reads what that one wrote.
template <typename K, typename... A>
inline cudaError_t launch_behind(K *kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------------------
// e4m3
// ---------------------------------------------------------------------------
// (lo, hi) -> two e4m3 bytes, nearest even, magnitudes above 448 clamped, NaN kept
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_from_e4m3x2(uint32_t b2) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)b2));
  return r;
}
__device__ __forceinline__ float2 f32x2_from_e4m3x2(uint32_t b2) {
  const uint32_t h = f16x2_from_e4m3x2(b2);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// not 0 where one of 16 e4m3 bytes is NaN (0x7f or 0xff)
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t nan_bytes(const uint4 &v) {
  return nan_bytes(v.x) | nan_bytes(v.y) | nan_bytes(v.z) | nan_bytes(v.w);
}

// Exponent k of the smallest power of two with amax <= 448 * 2^k (448 = 1.75
// * 2^8, the largest e4m3 value); amax is finite and not negative.
__device__ __forceinline__ int scale_exponent(float amax, int least = kMinScaleExp) {
  const uint32_t u = __float_as_uint(amax);
  const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(k, least);
}
__device__ __forceinline__ float exp2_int(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// ---------------------------------------------------------------------------
// block-wide exclusive scan of one long long per thread
// ---------------------------------------------------------------------------
// `tmp` holds 33 values; every thread of the block calls it.
__device__ __forceinline__ long long block_scan(long long v, long long *tmp, long long &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // tmp may still be read from the previous scan
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const long long w = lane < nw ? tmp[lane] : 0;
    long long s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    tmp[lane] = s - w;
    if (lane == 31) tmp[32] = s;
  }
  __syncthreads();
  total = tmp[32];
  return x - v + tmp[warp];
}

// ---------------------------------------------------------------------------
// the schedule of the attention over the cache
// ---------------------------------------------------------------------------
// A group is what shares a stream of keys: up to P consecutive query positions
// of one request and one slice of up to HS heads, its columns c = p * HS + h.
// The group's keys are pages (cache blocks): those of the raw rows its window
// reaches, then those of its completed compressed entries; a tile is the next
// 128 / bs of them.  All tiles of all groups form one line; CTA c works on
// tiles [c * quota, (c + 1) * quota) of it.  A group inside one CTA's range is
// written out directly, one that crosses ranges leaves a partial result (O, its
// reference exponent and its sum) in each CTA it touches, joined by the combine
// kernel.
struct __align__(16) Group {
  int tile0;        // first tile in the line
  int ntiles;
  int r;            // request
  int row0;         // row of the first position in q / out
  int pos0, npos;   // first position, positions
  int slice;        // head slice
  int pad;
};

// A CTA's piece of a group.
struct __align__(16) Segment {
  int r, row0, pos0, npos;
  int j0, j1;       // tiles of the group
  int slot;         // partial result slot, -1: the group is all here
  int slice_last;   // 2 * head slice + (the CTA's last segment)
  __device__ __forceinline__ int slice() const { return slice_last >> 1; }
  __device__ __forceinline__ bool last() const { return slice_last & 1; }
};

// What the combine kernel has to join at the border behind CTA c, written by
// that CTA: a group that begins in its range and ends behind it.
struct __align__(16) Border {
  int row;      // row of column 0 in out and lse, columns are rows in order
  int columns;  // 0: nothing to join
  int parts;
  int slot;     // of the first part; the others have slot 2 (c + i)
};

// The line has less than 2^31 tiles, or the call is refused.
constexpr long long kMaxTiles = 0x7fff0000ll;

struct SchedHeader {  // at the start of the workspace
  int32_t status;
  int32_t ngroups;
  int32_t ntiles;     // -1: refused, the attention fills its outputs with NaN
  int32_t longest;    // tiles of the longest group
};

// Many short groups (prompts): the line is cut between groups, which saves every
// CTA a partial group's beginning and end and the join (12 prompts of 200 to 500
// tokens over up to 130,000 rows, groups of up to 11 tiles: 152 us, 188 when cut
// anywhere); a group then counts for kGroupCost tiles more than it has, what its
// beginning and end take (0 and 4: 174 and 162 us).  Longer groups leave the CTAs
// less even than cuts cost (3 and 6 prompts of 447 tokens over 80,000 rows, groups
// of 43 tiles: 226 and 425 us cut anywhere, 276 and 457 cut between groups),
// unless a CTA has many of them (24 such prompts over up to 130,000 rows: 1,764 us,
// 1,363 cut between groups, which the rule leaves).
constexpr int kGroupCost = 2, kShortGroup = 32;

struct Pages {
  int rp0, nraw;  // first raw page, raw pages
  int ncomp;      // compressed pages
  int cp0;        // the first of them
};

__device__ __forceinline__ Pages group_pages(int pos0, int npos, int W, int m, int log_bs, bool comp) {
  Pages g;
  const int last = pos0 + npos - 1;
  g.rp0 = max(0, pos0 - W + 1) >> log_bs;
  g.nraw = (last >> log_bs) - g.rp0 + 1;
  const int ent = comp ? (last + 1) / m : 0;
  g.ncomp = (ent + (1 << log_bs) - 1) >> log_bs;
  g.cp0 = 0;
  return g;
}

// tiles per CTA
__device__ __forceinline__ int cta_quota(int ntiles, int grid, int min_tiles) {
  return max((int)(((uint32_t)max(ntiles, 0) + grid - 1) / (uint32_t)grid), min_tiles);
}

// Index of the group that holds tile t (all lanes of a warp call it): a search
// that narrows 32-fold a step, since each step is one dependent load.
// With `cost`, the line has so many places more in front of each later group.
__device__ __forceinline__ int find_group(const Group *groups, int n, int t, int cost = 0) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // groups[lo].tile0 <= t, hi is past the answer
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const bool le = i < hi && groups[i].tile0 + cost * i <= t;
    const uint32_t b = __ballot_sync(0xffffffffu, le);
    const int k = 31 - __clz(b);  // lane 0 always holds
    hi = min(hi, lo + (k + 1) * step);
    lo = lo + k * step;
  }
  return lo;
}

// Where a key lies among a group's columns: the columns [ca, cb) see it.
// Positions are group-relative; a raw row t is seen by t .. t + W - 1, a
// compressed entry j from its window's last position (j + 1) m - 1 on.
__device__ __forceinline__ void key_columns(bool comp, long long key, int pos0, int npos, int HS, int W, int m, int &ca,
                                            int &cb) {
  const long long from = comp ? (key + 1) * m - 1 - pos0 : key - pos0;
  const long long to = comp ? (long long)npos : from + W;  // exclusive
  const int a = (int)min(max(from, 0ll), (long long)npos), b = (int)min(max(to, 0ll), (long long)npos);
  ca = a * HS;
  cb = b * HS;
}

}  // namespace cache
}  // namespace hca
