// hca_cache_attn.cuh -- parameters of the attention-over-cache kernels.
#pragma once

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
};

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
__device__ __forceinline__ bool request_chunks(const AttnParams &p, int r, int &n) {
  const int s0 = p.start[r], s1 = p.start[r + 1], h = p.held[r];
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= p.N && h >= 0 && h <= kMaxPos - (s1 - s0) && (r > 0 || s0 == 0);
  n = ok ? (s1 - s0 + p.P - 1) / p.P : 0;
  return ok;
}

// Group of chunk c, the k-th of request r; false: the tables are too narrow.
__device__ __forceinline__ bool chunk_group(const AttnParams &p, int r, int k, Group &g) {
  const int s0 = p.start[r], T = p.start[r + 1] - s0, h = p.held[r], first = k * p.P;
  g.r = r;
  g.row0 = s0 + first;
  g.pos0 = h + first;
  g.npos = min(p.P, T - first);
  g.slice = 0;
  const Pages pg = group_pages(g.pos0, g.npos, p.W, p.m, p.log_bs, p.comp.table != nullptr);
  g.ntiles = (int)((((uint32_t)(pg.nraw + pg.ncomp) << p.log_bs) + kTileKeys - 1) / kTileKeys);
  // the raw table keeps the last cols pages of the request's tokens
  return ((h + T - 1) >> p.log_bs) - pg.rp0 < p.raw.cols && pg.ncomp <= p.comp.cols;
}

// tensor-core kernel (hca_cache_attn_tc.cu)
int tc_cache_ctas();     // CTAs per SM
int tc_cache_threads();  // threads of a CTA
cudaError_t tc_cache_attn(const AttnParams &p, cudaStream_t st);

}  // namespace cache
}  // namespace hca
