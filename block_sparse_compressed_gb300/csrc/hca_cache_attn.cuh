// hca_cache_attn.cuh -- parameters of the attention-over-cache kernels.
#pragma once

#include "hca_cache.cuh"

namespace hca {
namespace cache {

// CTAs of a launch, at most (the workspace holds two partial results for each)
inline int max_ctas(int NQ, bool tensor_cores) { return !tensor_cores ? 640 : NQ == 128 ? 160 : 320; }
constexpr int kSimtCols = 16;   // columns of an fp32 group
constexpr int kMinTiles = 2;    // fewest tiles a CTA takes (a partial result costs about as much as a tile)

struct AttnParams {
  const void *q;
  const int32_t *start, *held;
  CacheSet raw, comp;
  void *out;
  float *lse;
  SchedHeader *hdr;
  Group *groups;
  int32_t *gbase;      // [R + 1] first group (before slicing) of each request
  int32_t *first;      // [grid] group of each CTA's first tile
  float2 *part_ml;     // [2 * grid][NQ] reference exponent and sum of a partial result
  float *part_o;       // [2 * grid][NQ][D]
  int N, R, H, D, W, m, log_bs;
  int HS, slices, P;   // heads per slice, slices, positions per group
  int NQ;              // columns of a group, P * HS <= NQ
  int grid;            // CTAs of the attention kernel
  float scale;
  uint64_t wait_ns;
  int stall;
};

// Columns of a group that stand for a (position, head).
__device__ __forceinline__ int real_columns(const AttnParams &p, const Group &g) {
  return p.P == 1 ? min(p.HS, p.H - g.slice * p.HS) : g.npos * p.HS;
}

// A CTA's piece of a group: tiles [j0, j1) of it.
struct Segment {
  int j0, j1;
  bool whole;  // all of the group's tiles
  int slot;    // partial result slot otherwise
};
__device__ __forceinline__ Segment segment_of(const Group &g, long long c0, long long c1, int cta) {
  Segment s;
  const long long a = g.tile0 > c0 ? g.tile0 : c0, b = min(g.tile0 + g.ntiles, c1);
  s.j0 = (int)(a - g.tile0);
  s.j1 = (int)(b - g.tile0);
  s.whole = s.j0 == 0 && s.j1 == g.ntiles;
  // the group that enters the CTA's range from before it takes slot 0
  s.slot = 2 * cta + (a == c0 ? 0 : 1);
  return s;
}

// tensor-core kernel (hca_cache_attn_tc.cu)
int tc_cache_ctas(int NQ);  // CTAs per SM
cudaError_t tc_cache_attn(const AttnParams &p, cudaStream_t st);

}  // namespace cache
}  // namespace hca
