// hca_cache_attn.cu -- attention over the 8-bit cache: the schedule of its
// tiles, the fp32 kernel and the join of partial results.
//
// Query position i of a request attends under one softmax to the raw rows
// i - W < t <= i and the compressed entries (j + 1) m <= i + 1 of its request,
// read from cache blocks through block tables.  A key of block b is
// s_b * k8 with e4m3 values k8, so its score is scale * s_b * <q, k8> and its
// part of the output p * s_b * k8: the values are used as they lie in memory
// and the scale multiplies one number for each key.
//
// Few rows and long caches leave most SMs idle unless the keys are divided, so
// all tiles of all groups (hca_cache.cuh) are laid out as one line and cut into
// equal ranges; a group cut by a range border is joined by the combine kernel
// from each part's (O, reference exponent, sum).
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "hca_cache_attn.cuh"
#include "tc_tiles.cuh"

namespace hca {
using namespace cache;

namespace {

// ---------------------------------------------------------------------------
// schedule
// ---------------------------------------------------------------------------
constexpr int kSchedThreads = 1024;

template <typename P>
__global__ void __launch_bounds__(kSchedThreads) hca_cache_sched_kernel(const P p) {
  __shared__ long long tmp[33];
  __shared__ int longest;
  const int tid = threadIdx.x;
  if (tid == 0) longest = 0;
  tc::pdl_launch_dependents();  // the attention kernel waits for this one's end by itself
  bool ok = prefixes_ok(p);
  long long chunks = 0;
  for (int r0 = 0; r0 < p.R; r0 += kSchedThreads) {
    const int r = r0 + tid;
    int n = 0;
    if (r < p.R) ok = request_chunks(p, r, n) && ok;
    long long all;
    const long long before = block_scan(n, tmp, all);
    if (r < p.R) p.gbase[r] = (int)(chunks + before);
    chunks += all;
  }
  if (tid == 0) p.gbase[p.R] = (int)chunks;
  ok = __syncthreads_and(ok);
  if (!ok) chunks = 0;
  long long line = 0;
  for (long long c0 = 0; c0 < chunks; c0 += kSchedThreads) {
    const long long c = c0 + tid;
    Group g;
    g.ntiles = 0;
    if (c < chunks) {
      int lo = 0, hi = p.R;  // gbase[lo] <= c < gbase[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.gbase[mid] <= c) lo = mid; else hi = mid;
      }
      ok = chunk_group(p, lo, (int)c - p.gbase[lo], g) && ok;
      atomicMax(&longest, g.ntiles);
    }
    long long all;
    const long long before = block_scan(g.ntiles, tmp, all);
    if (c < chunks) {
      for (int s = 0; s < p.slices; ++s) {
        g.slice = s;
        g.tile0 = (int)((line + before) * p.slices + (long long)s * g.ntiles);  // of use if all of it fits
        p.groups[c * p.slices + s] = g;
      }
    }
    line += all;
  }
  ok = __syncthreads_and(ok) && line * p.slices < kMaxTiles;
  if (tid == 0) {
    p.hdr->ngroups = (int)(chunks * p.slices);
    p.hdr->ntiles = ok ? (int)(line * p.slices) : -1;
    p.hdr->longest = longest;
  }
}

// ---------------------------------------------------------------------------
// helpers of the fp32 kernel
// ---------------------------------------------------------------------------
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void put4(float *p, const float4 &v, float f) {
  *reinterpret_cast<float4 *>(p) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ void put4(__nv_bfloat16 *p, const float4 &v, float f) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(tc::pack_bf16x2(v.x * f, v.y * f), tc::pack_bf16x2(v.z * f, v.w * f));
}

// Every output of a call that failed on the device is NaN.
template <typename T>
__device__ __forceinline__ void poison(const AttnParams &p) {
  const size_t n = (size_t)p.N * p.H;
  const float nan = __int_as_float(0x7fc00000);
  const size_t at = ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x;
  const size_t step = (size_t)gridDim.y * gridDim.x * blockDim.x;
  for (size_t i = at; i < n * p.D; i += step)
    put(static_cast<T *>(p.out) + i, nan);
  for (size_t i = at; i < n; i += step)
    p.lse[i] = nan;
}

// ---------------------------------------------------------------------------
// fp32 kernel: one thread per key for the scores, one per dimension for the
// output; D a multiple of 16 up to 256.  Rows of q share a key tile in groups of
// kCols; of more columns than the requests' tokens fill the rest is wasted (8
// requests of one or two tokens and 4 heads over up to 4,000 rows: 17.2 us with 8
// columns, 20.6 with 16).  Bound by latency: the tile's table, scale and rows are
// three dependent loads.
// ---------------------------------------------------------------------------
constexpr int kSimtThreads = 128;

template <int kCols>
struct SimtShared {
  float q[256][kCols];                // [d][c]
  float pr[kTileKeys][kCols];         // probabilities times the block's scale
  float red[4][kCols];
  float m[kCols], f[kCols], l[kCols];
  const uint8_t *rows[8];             // the tile's pages (NULL: none, or a bad block id or scale)
  float scale[8];
  int key0[8], kind[8];               // kind 0 raw, 1 compressed, 2 no page
  int first;
  Group groups[kSimtThreads];         // the line's, where this kernel works them out
  int gbase[kSimtThreads];
  long long tmp[33];
};

// The line's groups by the CTA's threads, one each, into sh.groups; returns its
// tiles (-1: refused).
template <typename P, int kCols>
__device__ __forceinline__ int schedule(const P &p, SimtShared<kCols> &sh, int &ngroups) {
  const int tid = threadIdx.x;
  int n = 0;
  bool ok = prefixes_ok(p);
  if (tid < p.R) ok = request_chunks(p, tid, n) && ok;
  long long chunks, tiles;
  sh.gbase[tid] = (int)block_scan(n, sh.tmp, chunks);
  ok = __syncthreads_and(ok);
  Group g;
  g.ntiles = 0;
  const bool mine = ok && tid < chunks;
  if (mine) {
    int lo = 0, hi = p.R;  // gbase[lo] <= tid < gbase[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sh.gbase[mid] <= tid) lo = mid; else hi = mid;
    }
    ok = chunk_group(p, lo, tid - sh.gbase[lo], g);
  }
  g.tile0 = (int)block_scan(g.ntiles, sh.tmp, tiles);
  if (mine) sh.groups[tid] = g;
  ngroups = (int)chunks;
  return __syncthreads_and(ok) && tiles < kMaxTiles ? (int)tiles : -1;
}

template <int kCols, typename P>
__global__ void __launch_bounds__(kSimtThreads) hca_cache_simt_kernel(const P p) {
  extern __shared__ uint8_t keys[];  // [128][D + 4] bytes: a row's words fall into different banks
  __shared__ SimtShared<kCols> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int ntiles, ngroups;
  if (p.in_cta) {
    ntiles = schedule(p, sh, ngroups);
  } else {
    tc::pdl_wait();
    ntiles = p.hdr->ntiles;
    ngroups = p.hdr->ngroups;
  }
  const Group *groups = p.in_cta ? sh.groups : p.groups;
  tc::pdl_launch_dependents();
  if (tid == 0) {
    p.err[blockIdx.x] = ntiles < 0 ? HCA_ERR_CACHE : HCA_OK;
    p.border[blockIdx.x] = Border{0, 0, 0, 0};
  }
  if (ntiles < 0) {
    poison<float>(p);
    return;
  }
  const int quota = cta_quota(ntiles, p.grid, p.min_tiles);
  if (blockIdx.x >= (ntiles + quota - 1) / quota) return;
  const int c0 = quota * blockIdx.x, c1 = min(c0 + quota, ntiles);
  if (warp == 0) {
    const int g = find_group(groups, ngroups, c0);
    if (lane == 0) sh.first = g;
  }
  __syncthreads();
  int gi = sh.first;
  const int pitch = p.D + 4, upr = p.D / 4, ppt = kTileKeys >> p.log_bs, off = tid & ((1 << p.log_bs) - 1);
  // output threads: dimension d, keys k0, k0 + kstep, ...
  int dpad = 16;
  while (dpad < p.D && dpad < kSimtThreads) dpad *= 2;
  const int kstep = kSimtThreads / dpad, kfirst = tid / dpad;
  for (bool last = false; !last; ++gi) {
    __syncthreads();
    const Group g = groups[gi];
    const Segment seg = segment_of(g, c0, c1, blockIdx.x);
    last = seg.last();
    if (last && tid == 0) p.border[blockIdx.x] = border_of(p, g, c0, c1, quota, blockIdx.x);
    const int nreal = real_columns(p, g.npos, g.slice);
    const size_t row0 = (size_t)g.row0 * p.H + g.slice * p.HS;  // columns are rows of q and out in order
    const Pages pg = group_pages(g.pos0, g.npos, p.W, p.m, p.log_bs, p.comp.table != nullptr);
#pragma unroll 4
    for (int i = tid; i < p.D * kCols; i += kSimtThreads) {
      const int c = i / p.D, d = i % p.D;
      sh.q[d][c] = c < nreal ? static_cast<const float *>(p.q)[row0 * p.D + i] : 0.f;
    }
    if (tid < kCols) {
      sh.m[tid] = -INFINITY;
      sh.l[tid] = 0.f;
    }
    float o[2][kCols];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[x][c] = 0.f;
    const float sl2 = p.scale * 1.4426950408889634f;
    for (int j = seg.j0; j < seg.j1; ++j) {
      __syncthreads();
      if (tid < ppt) {
        const int v = j * ppt + tid;
        sh.rows[tid] = nullptr;
        sh.scale[tid] = __int_as_float(0x7fc00000);
        sh.kind[tid] = 2;
        if (v < pg.nraw + pg.ncomp) {
          const bool comp = v >= pg.nraw;
          const CacheSet &s = comp ? p.comp : p.raw;
          const int page = comp ? v - pg.nraw : pg.rp0 + v;
          sh.kind[tid] = comp;
          sh.key0[tid] = page << p.log_bs;
          const int id = s.table[(size_t)g.r * s.cols + page % s.cols];
          const float sc = id >= 0 && id < s.nblocks ? s.scale[id] : 0.f;
          if (sc > 0.f && sc < INFINITY) {
            sh.rows[tid] = s.pool + ((size_t)id << p.log_bs) * p.D;
            sh.scale[tid] = sc;
          } else {
            p.err[blockIdx.x] = HCA_ERR_CACHE;
          }
        }
      }
      __syncthreads();
      // stage the tile's rows, 16 bytes at a time and 4 loads in flight
      const int u16 = p.D / 16, units = kTileKeys * u16;
      for (int i0 = tid; i0 < units; i0 += 4 * kSimtThreads) {
        uint4 w[4];
        int row[4], u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = i0 + k * kSimtThreads;
          row[k] = i / u16;
          u[k] = i - row[k] * u16;
          const uint8_t *rows = i < units ? sh.rows[row[k] >> p.log_bs] : nullptr;
          w[k] = make_uint4(0, 0, 0, 0);
          if (rows) w[k] = reinterpret_cast<const uint4 *>(rows + (size_t)(row[k] & ((1 << p.log_bs) - 1)) * p.D)[u[k]];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (i0 + k * kSimtThreads >= units) break;
          uint32_t *to = reinterpret_cast<uint32_t *>(keys + row[k] * pitch + 16 * u[k]);
          to[0] = w[k].x; to[1] = w[k].y; to[2] = w[k].z; to[3] = w[k].w;
        }
      }
      const int kind = sh.kind[tid >> p.log_bs];
      const float sk = sh.scale[tid >> p.log_bs];
      int ca = 0, cb = 0;
      if (kind < 2) key_columns(kind == 1, (long long)sh.key0[tid >> p.log_bs] + off, g.pos0, g.npos, p.HS, p.W, p.m, ca, cb);
      __syncthreads();
      float s[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) s[c] = 0.f;
#pragma unroll 2
      for (int u = 0; u < upr; ++u) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(keys + tid * pitch + 4 * u);
        const float2 a = f32x2_from_e4m3x2(w & 0xffffu), b = f32x2_from_e4m3x2(w >> 16);
        const float kk[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int c = 0; c < kCols; ++c) s[c] = fmaf(kk[e], sh.q[4 * u + e][c], s[c]);
      }
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        // a masked key's row may hold anything, NaN among it
        s[c] = c >= ca && c < cb ? s[c] * (sl2 * sk) : -INFINITY;
        float mx = s[c];
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        if (lane == 0) sh.red[warp][c] = mx;
      }
      __syncthreads();
      if (tid < kCols) {
        const float mx = fmaxf(fmaxf(sh.red[0][tid], sh.red[1][tid]), fmaxf(sh.red[2][tid], sh.red[3][tid]));
        const float mo = sh.m[tid], mn = fmaxf(mo, mx);
        sh.f[tid] = mn == -INFINITY ? 1.f : exp2f(mo - mn);
        sh.m[tid] = mn;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const float mn = sh.m[c];
        const float e = s[c] == -INFINITY ? 0.f : exp2f(s[c] - mn);
        sh.pr[tid][c] = e == 0.f ? 0.f : e * sk;
        float sum = e;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        if (lane == 0) sh.red[warp][c] = sum;
      }
      bool clear = cb <= ca;
      if (!clear && cb - ca < g.npos * p.HS) {
        uint32_t nan = 0;
        for (int u = 0; u < upr; ++u) nan |= nan_bytes(*reinterpret_cast<const uint32_t *>(keys + tid * pitch + 4 * u));
        clear = nan != 0;
      }
      if (clear) {
        // its values meet a probability of 0, where 0 * NaN is not 0; a column
        // that sees a NaN has one for a probability
        for (int u = 0; u < upr; ++u) *reinterpret_cast<uint32_t *>(keys + tid * pitch + 4 * u) = 0;
      }
      __syncthreads();
      if (tid < kCols)
        sh.l[tid] = sh.l[tid] * sh.f[tid] + ((sh.red[0][tid] + sh.red[1][tid]) + (sh.red[2][tid] + sh.red[3][tid]));
#pragma unroll
      for (int x2 = 0; x2 < 2; ++x2) {
        const int d = tid % dpad + x2 * kSimtThreads;
        if (d >= p.D) break;
        float acc[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
#pragma unroll 8
        for (int k = kfirst; k < kTileKeys; k += kstep) {
          const float v = f32x2_from_e4m3x2(keys[k * pitch + d]).x;
#pragma unroll
          for (int c = 0; c < kCols; ++c) acc[c] = fmaf(sh.pr[k][c], v, acc[c]);
        }
#pragma unroll
        for (int c = 0; c < kCols; ++c) o[x2][c] = fmaf(o[x2][c], sh.f[c], acc[c]);
      }
    }
    __syncthreads();
    // join the key subsets of a dimension (D < 128), then write
    float *join = &sh.pr[0][0];  // [kstep][dpad][kCols]
    if (kstep > 1) {
#pragma unroll
      for (int c = 0; c < kCols; ++c) join[tid * kCols + c] = o[0][c];
      __syncthreads();
      if (kfirst == 0)
        for (int k = 1; k < kstep; ++k)
#pragma unroll
          for (int c = 0; c < kCols; ++c) o[0][c] += join[(k * dpad + tid) * kCols + c];
    }
#pragma unroll
    for (int x2 = 0; x2 < 2; ++x2) {
      const int d = tid % dpad + x2 * kSimtThreads;
      if (d >= p.D || (kstep > 1 && kfirst > 0)) continue;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        if (c >= nreal) continue;
        if (seg.slot < 0) static_cast<float *>(p.out)[(row0 + c) * p.D + d] = o[x2][c] / sh.l[c];
        else p.part_o[((size_t)seg.slot * kCols + c) * p.D + d] = o[x2][c];
      }
    }
    if (seg.slot >= 0 && tid == 0) p.part_unit[seg.slot] = 0;
    if (tid < nreal) {
      if (seg.slot < 0) p.lse[row0 + tid] = (sh.m[tid] + log2f(sh.l[tid])) * 0.69314718055994531f;
      else p.part_ml[(size_t)seg.slot * kCols + tid] = make_float2(sh.m[tid], sh.l[tid]);
    }
  }
}

// ---------------------------------------------------------------------------
// combine: out = sum 2^(m_i - M + u_i) O_i / sum 2^(m_i - M) l_i over a group's
// parts, whose O_i have units of 2^u_i, and the call's status from its CTAs'
// ---------------------------------------------------------------------------
constexpr int kCombineWarps = 8, kCombineThreads = 32 * kCombineWarps;
constexpr int kMaxBorders = 640;

// 2^(unit - largest), what a part's O counts beside one of the largest unit
__device__ __forceinline__ float unit_weight(int unit, int largest) { return exp2_int(max(unit - largest, -126)); }

// The call's status from its CTAs' ones, written by the grid's first block; true
// if a wait gave up: the outputs become NaN.
template <typename T>
__device__ __forceinline__ bool settle_status(const AttnParams &p) {
  int worst = HCA_OK;
  for (int i = threadIdx.x; i < p.grid; i += kCombineThreads) worst = max(worst, p.err[i] == HCA_ERR_TIMEOUT ? 1000 : p.err[i]);
  const bool late = __syncthreads_or(worst == 1000);
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    const bool bad = __syncthreads_or(worst != HCA_OK);
    if (threadIdx.x == 0) p.hdr->status = late ? HCA_ERR_TIMEOUT : bad ? HCA_ERR_CACHE : HCA_OK;
  }
  if (late) poison<T>(p);
  return late;
}

// Many groups: block (c, y) joins 32 columns of the group that begins in CTA c's
// range and ends behind it.  8 lanes have a column, kX float4 of it each, so that
// a warp's loads of 4 columns are in flight together.
template <typename T, int kX>
__global__ void __launch_bounds__(kCombineThreads, 4) hca_cache_combine_kernel(const AttnParams p) {
  tc::pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l8 = lane & 7;
  const Border g = p.border[blockIdx.x];
  if (g.columns <= (int)blockIdx.y * 4 * kCombineWarps) {
    settle_status<T>(p);
    return;
  }
  const int c = (blockIdx.y * kCombineWarps + warp) * 4 + (lane >> 3);
  const bool mine = c < g.columns;
  const int n = g.parts, v4 = p.D / 4;
  auto part = [&](int i) { return i == 0 ? g.slot : 2 * ((int)blockIdx.x + i); };
  auto slot = [&](int i) { return (size_t)part(i) * p.NQ + c; };
  float M = -INFINITY, L = 0.f;
  int U = INT_MIN;
  for (int i = l8; mine && i < n; i += 8) {
    const float2 ml = p.part_ml[slot(i)];
    M = fmaxf(M, ml.x);
    if (ml.y != 0.f) U = max(U, p.part_unit[part(i)]);  // 0: a part in which the column saw no key
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    U = max(U, __shfl_xor_sync(0xffffffffu, U, o));
  }
  float4 acc[kX];
#pragma unroll
  for (int x = 0; x < kX; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int b = 0; b < n; b += 8) {
    float w = 0.f;
    if (mine && b + l8 < n) {
      const float2 ml = p.part_ml[slot(b + l8)];
      if (ml.y != 0.f) {
        w = exp2f(ml.x - M);
        L += w * ml.y;
        w *= unit_weight(p.part_unit[part(b + l8)], U);
      }
    }
    const int k1 = min(8, n - b);
#pragma unroll 2
    for (int k = 0; k < k1; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, (lane & 24) | k);
      const float4 *o = reinterpret_cast<const float4 *>(p.part_o + slot(b + k) * p.D);
      if (mine && wk != 0.f) {
#pragma unroll
        for (int x = 0; x < kX; ++x) {
          if (l8 + 8 * x < v4) {
            const float4 v = o[l8 + 8 * x];
            acc[x].x = fmaf(wk, v.x, acc[x].x); acc[x].y = fmaf(wk, v.y, acc[x].y);
            acc[x].z = fmaf(wk, v.z, acc[x].z); acc[x].w = fmaf(wk, v.w, acc[x].w);
          }
        }
      }
    }
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  // the statuses' latency passes behind the parts'
  if (settle_status<T>(p) || !mine) return;
  const float inv = exp2_int(U) / L;
  const size_t row = (size_t)g.row + c;
#pragma unroll
  for (int x = 0; x < kX; ++x)
    if (l8 + 8 * x < v4) put4(static_cast<T *>(p.out) + row * p.D + 4 * (l8 + 8 * x), acc[x], inv);
  if (l8 == 0) p.lse[row] = (M + log2f(L)) * 0.69314718055994531f;
}

// Few groups (few rows over long caches): a group has many parts, so several
// warps share a column's; the joins are listed by every block, as their places
// among the borders are not known, and dealt out column by column.
__device__ __forceinline__ int warps_per_column(int parts) { return parts >= 32 ? 8 : parts >= 16 ? 4 : parts >= 8 ? 2 : 1; }

template <typename T>
__global__ void __launch_bounds__(kCombineThreads) hca_cache_combine_few_kernel(const AttnParams p) {
  __shared__ float4 acc[kCombineWarps][64];
  __shared__ int before[kMaxBorders + 1];
  __shared__ long long tmp[33];
  tc::pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (settle_status<T>(p)) return;
  const int per = (p.grid + kCombineThreads - 1) / kCombineThreads, i0 = tid * per, i1 = min(i0 + per, p.grid);
  int items = 0;
  for (int i = i0; i < i1; ++i) {
    const Border g = p.border[i];
    before[i] = items;
    if (g.columns > 0) items += (g.columns * warps_per_column(g.parts) + kCombineWarps - 1) / kCombineWarps;
  }
  long long total;
  const int base = (int)block_scan(items, tmp, total);
  for (int i = i0; i < i1; ++i) before[i] += base;
  __syncthreads();
  const int v4 = p.D / 4;  // float4 of a row, at most 64
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int lo = 0, hi = p.grid;  // before[lo] <= item < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= item) lo = mid; else hi = mid;
    }
    const Border g = p.border[lo];
    const int wpc = warps_per_column(g.parts);
    const int c = (item - before[lo]) * (kCombineWarps / wpc) + warp / wpc, sub = warp % wpc;
    const int n = c < g.columns ? g.parts : 0;
    auto slot = [&](int i) { return (size_t)(i == 0 ? g.slot : 2 * (lo + i)); };
    float M = -INFINITY, L = 0.f;
    int U = INT_MIN;
    for (int i = lane; i < n; i += 32) {
      const float2 ml = p.part_ml[slot(i) * p.NQ + c];
      M = fmaxf(M, ml.x);
      if (ml.y != 0.f) U = max(U, p.part_unit[slot(i)]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    U = __reduce_max_sync(0xffffffffu, U);
    float4 s[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int b = 0; b < n; b += 32) {
      float w = 0.f;
      if (b + lane < n) {
        const float2 ml = p.part_ml[slot(b + lane) * p.NQ + c];
        if (ml.y != 0.f) {
          w = exp2f(ml.x - M);
          L += w * ml.y;
          w *= unit_weight(p.part_unit[slot(b + lane)], U);
        }
      }
      const int k1 = min(32, n - b);
#pragma unroll 4
      for (int k = sub; k < k1; k += wpc) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        const float4 *o = reinterpret_cast<const float4 *>(p.part_o + (slot(b + k) * p.NQ + c) * p.D);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (lane + 32 * x < v4 && wk != 0.f) {
            const float4 v = o[lane + 32 * x];
            s[x].x = fmaf(wk, v.x, s[x].x); s[x].y = fmaf(wk, v.y, s[x].y);
            s[x].z = fmaf(wk, v.z, s[x].z); s[x].w = fmaf(wk, v.w, s[x].w);
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    __syncthreads();
    acc[warp][lane] = s[0];
    acc[warp][32 + lane] = s[1];
    __syncthreads();
    for (int w = 1; sub == 0 && w < wpc; ++w) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float4 u = acc[warp + w][lane + 32 * x];
        s[x].x += u.x; s[x].y += u.y; s[x].z += u.z; s[x].w += u.w;
      }
    }
    if (n > 0 && sub == 0) {
      const float inv = exp2_int(U) / L;
      const size_t row = (size_t)g.row + c;
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (lane + 32 * x < v4) put4(static_cast<T *>(p.out) + row * p.D + 4 * (lane + 32 * x), s[x], inv);
      if (lane == 0) p.lse[row] = (M + log2f(L)) * 0.69314718055994531f;
    }
  }
}

template <int kCols, typename P>
cudaError_t simt(const P &p, cudaStream_t st) {
  static tc::SmemAttrOnce attr;
  const cudaError_t e = attr.ensure(reinterpret_cast<const void *>(hca_cache_simt_kernel<kCols, P>), kTileKeys * (256 + 4));
  if (e != cudaSuccess) return e;
  ProfScope prof(kKCacheSimt, st);
  if (!p.in_cta) return launch_behind(hca_cache_simt_kernel<kCols, P>, dim3(p.grid), kSimtThreads, kTileKeys * (p.D + 4), st, p);
  hca_cache_simt_kernel<kCols, P><<<p.grid, kSimtThreads, kTileKeys * (p.D + 4), st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t combine(const AttnParams &p, int gmax, int sms, cudaStream_t st) {
  // Few groups: fewer than leave each 16 CTAs.  One, 8, 16 and 19 requests over 100,000
  // rows at m = 4 take 26.7, 33.0, 41.8 and 47.2 us, with the kernel of many groups
  // 62.2, 43.6, 46.6 and 48.7; 24 and 48 52.8 and 80.7, with the one of few 53.2 and
  // 83.8.
  const bool few = (long long)gmax * 16 <= p.grid;
  const dim3 grid = few ? dim3(4 * sms) : dim3(p.grid, (p.P * p.HS + 4 * kCombineWarps - 1) / (4 * kCombineWarps));
  ProfScope prof(kKCacheCombine, st);
  // its blocks are set up while the attention's last CTAs run
  if (few) return launch_behind(hca_cache_combine_few_kernel<T>, grid, kCombineThreads, 0, st, p);
  if constexpr (std::is_same_v<T, float>) {  // bf16: D is 64 or 128
    if (p.D > 128) return launch_behind(hca_cache_combine_kernel<T, 8>, grid, kCombineThreads, 0, st, p);
  }
  return launch_behind(hca_cache_combine_kernel<T, 4>, grid, kCombineThreads, 0, st, p);
}

// Columns of a group for H heads: enough for one position's slice of heads, and
// for as many positions as the average request brings.  More columns share a
// key tile between more rows; unused ones cost tensor and exponential work.
bool on_tensor_cores(int dtype) { return dtype == HCA_BF16; }

int pick_columns(int N, int R, int H, int dtype) {
  const int most = on_tensor_cores(dtype) ? 128 : kSimtCols;
  const int slices = (H + most - 1) / most, HS = (H + slices - 1) / slices;
  const int T = R > 0 ? (N + R - 1) / R : 1;
  const long long want = (long long)HS * T;
  if (!on_tensor_cores(dtype)) return want <= 4 ? 4 : want <= 8 ? 8 : kSimtCols;
  return want <= 32 ? 32 : want <= 64 ? 64 : 128;
}

struct Layout {
  int NQ, HS, slices, P;
  size_t gmax;
  size_t off_gbase, off_groups, off_err, off_border, off_unit, off_ml, off_o, bytes;
  int ctas;  // at most
};

Layout layout_of(int N, int R, int H, int D, int dtype) {
  Layout l;
  l.NQ = pick_columns(N, R, H, dtype);
  const int most = on_tensor_cores(dtype) ? 128 : kSimtCols;
  l.slices = (H + most - 1) / most;
  l.HS = (H + l.slices - 1) / l.slices;
  l.P = l.slices == 1 ? l.NQ / l.HS : 1;
  // a request's last chunk may be short, and a chunk has at least one token
  l.gmax = std::min((size_t)N / l.P + R, (size_t)N) * l.slices;
  l.ctas = max_ctas(on_tensor_cores(dtype));
  const size_t slots = 2 * (size_t)l.ctas;
  size_t at = kHeaderBytes;
  l.off_gbase = at;
  at += align_up(((size_t)R + 1) * sizeof(int32_t));
  l.off_groups = at;
  at += align_up(l.gmax * sizeof(Group));
  l.off_err = at;
  at += align_up(l.ctas * sizeof(int32_t));
  l.off_border = at;
  at += align_up(l.ctas * sizeof(Border));
  l.off_unit = at;
  at += align_up(slots * sizeof(int32_t));
  l.off_ml = at;
  at += align_up(slots * l.NQ * sizeof(float2));
  l.off_o = at;
  at += align_up(slots * l.NQ * D * sizeof(float));
  l.bytes = at;
  return l;
}

int log2_int(int v) {
  int k = 0;
  while ((1 << k) < v) ++k;
  return k;
}

}  // namespace

size_t cache_attn_ws_bytes(int N, int R, int H, int D, int dtype) { return layout_of(N, R, H, D, dtype).bytes; }

long long cache_attn_groups(int N, int R, int H, int D, int dtype) { return (long long)layout_of(N, R, H, D, dtype).gmax; }

namespace {

// Parameters of a call's kernels; sms: SMs of the device.
void fill(AttnParams &p, const CacheAttnArgs &a, int sms) {
  const Layout l = layout_of(a.N, a.R, a.H, a.D, a.dtype);
  char *ws = static_cast<char *>(a.ws);
  p.q = a.q; p.start = a.start; p.held = a.held; p.raw = a.raw; p.comp = a.comp; p.out = a.out; p.lse = a.lse;
  p.hdr = reinterpret_cast<SchedHeader *>(ws);
  p.gbase = reinterpret_cast<int32_t *>(ws + l.off_gbase);
  p.groups = reinterpret_cast<Group *>(ws + l.off_groups);
  p.err = reinterpret_cast<int32_t *>(ws + l.off_err);
  p.border = reinterpret_cast<Border *>(ws + l.off_border);
  p.part_ml = reinterpret_cast<float2 *>(ws + l.off_ml);
  p.part_o = reinterpret_cast<float *>(ws + l.off_o);
  p.part_unit = reinterpret_cast<int32_t *>(ws + l.off_unit);
  p.N = a.N; p.R = a.R; p.H = a.H; p.D = a.D; p.W = a.W; p.m = a.m; p.log_bs = log2_int(a.bs);
  p.HS = l.HS; p.slices = l.slices; p.P = l.P; p.NQ = l.NQ;
  p.scale = a.scale; p.wait_ns = std::min<uint64_t>(a.wait_ns, 4000000000u); p.stall = a.stall;
  const bool tcs = on_tensor_cores(a.dtype);
  p.grid = std::min((tcs ? tc_cache_ctas() : 4) * sms, l.ctas);
  // a CTA of one tile costs a part to join (94 tokens of 37 requests: 20.6 us, 18.6 with 2, 20.4 with 4)
  p.min_tiles = tcs ? 2 : 1;
  const int threads = tcs ? tc_cache_threads() : kSimtThreads;
  p.in_cta = l.slices == 1 && a.R <= threads && l.gmax <= (size_t)threads;
}

template <typename P>
cudaError_t attend(P &p, const CacheAttnArgs &a, cudaStream_t st) {
  const Layout l = layout_of(a.N, a.R, a.H, a.D, a.dtype);
  const int sms = tc::sm_count();
  if (sms <= 0) return cudaErrorNoDevice;
  fill(p, a, sms);
  const bool tcs = on_tensor_cores(a.dtype);
  if (!p.in_cta) {
    ProfScope prof(kKCacheSched, st);
    hca_cache_sched_kernel<P><<<1, kSchedThreads, 0, st>>>(p);
  }
  if (tcs) {
    const cudaError_t e = tc_cache_attn(p, st);
    if (e != cudaSuccess) return e;
  } else {
    const cudaError_t e = p.NQ == 4 ? simt<4>(p, st) : p.NQ == 8 ? simt<8>(p, st) : simt<kSimtCols>(p, st);
    if (e != cudaSuccess) return e;
  }
  if constexpr (P::kShared) {
    if (p.joined) return cudaSuccess;
  }
  const int gmax = (int)std::min<size_t>(l.gmax, 1 << 20);
  const bool bf16_rows = tcs && !(P::kShared && a.share.apart);
  const cudaError_t e = bf16_rows ? combine<__nv_bfloat16>(p, gmax, sms, st) : combine<float>(p, gmax, sms, st);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t cache_attn(const CacheAttnArgs &a, cudaStream_t st) {
  if (a.share.G == 0) {
    AttnParams p;
    return attend(p, a, st);
  }
  SharedAttnParams p;
  shared_params(a, p);
  return attend(p, a, st);
}

void cache::shared_params(const CacheAttnArgs &a, SharedAttnParams &p) {
  p.sms = std::max(tc::sm_count(), 0);
  fill(p, a, p.sms);
  p.first = a.share.first; p.cols = a.share.cols; p.G = a.share.G; p.apart = a.share.apart;
  p.beside = a.share.beside && p.in_cta;
  p.joined = a.share.joined && p.beside;
}

}  // namespace hca
