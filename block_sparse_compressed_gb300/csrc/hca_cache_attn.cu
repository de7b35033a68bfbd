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

#include "hca_cache_attn.cuh"
#include "tc_tiles.cuh"

namespace hca {
using namespace cache;

namespace {

// ---------------------------------------------------------------------------
// schedule
// ---------------------------------------------------------------------------
constexpr int kSchedThreads = 1024;

__global__ void __launch_bounds__(kSchedThreads) hca_cache_sched_kernel(const AttnParams p) {
  __shared__ long long tmp[33];
  const int tid = threadIdx.x;
  const int bs = 1 << p.log_bs;
  // chunks of P positions of every request, and the checks of the lengths
  bool ok = p.start[0] == 0;
  long long chunks = 0;
  for (int r0 = 0; r0 < p.R; r0 += kSchedThreads) {
    const int r = r0 + tid;
    long long n = 0;
    if (r < p.R) {
      const long long s0 = p.start[r], s1 = p.start[r + 1], h = p.held[r];
      const long long T = s1 - s0;
      const bool good = T >= 0 && s0 >= 0 && s1 <= p.N && h >= 0 && h + T <= kMaxPos;
      ok = ok && good;
      if (good) n = (T + p.P - 1) / p.P;
    }
    long long all;
    const long long before = block_scan(n, tmp, all);
    if (r < p.R) p.gbase[r] = (int)(chunks + before);
    chunks += all;
  }
  if (tid == 0) p.gbase[p.R] = (int)chunks;
  ok = __syncthreads_and(ok);
  if (!ok) chunks = 0;
  // groups: a chunk's tiles, and its place in the line
  long long line = 0;
  bool fits = true;
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
      const int first = ((int)c - p.gbase[lo]) * p.P;
      const int T = p.start[lo + 1] - p.start[lo];
      const int h = p.held[lo];
      g.r = lo;
      g.row0 = p.start[lo] + first;
      g.pos0 = h + first;
      g.npos = min(p.P, T - first);
      const Pages pg = group_pages(g.pos0, g.npos, p.W, p.m, p.log_bs, p.comp.table != nullptr);
      g.ntiles = (int)(((long long)(pg.nraw + pg.ncomp) * bs + kTileKeys - 1) / kTileKeys);
      // the raw table keeps the last cols pages of the request's tokens
      fits = fits && ((h + T - 1) >> p.log_bs) - pg.rp0 < p.raw.cols && pg.ncomp <= p.comp.cols;
    }
    long long all;
    const long long before = block_scan(g.ntiles, tmp, all);
    if (c < chunks) {
      for (int s = 0; s < p.slices; ++s) {
        g.slice = s;
        g.tile0 = (line + before) * p.slices + (long long)s * g.ntiles;
        p.groups[c * p.slices + s] = g;
      }
    }
    line += all;
  }
  fits = __syncthreads_and(fits);
  if (tid == 0) {
    p.hdr->status = ok && fits ? HCA_OK : HCA_ERR_CACHE;
    p.hdr->ngroups = (int)(chunks * p.slices);
    p.hdr->ntiles = ok && fits ? line * p.slices : -1;  // -1: the attention fills its outputs with NaN
  }
}

// ---------------------------------------------------------------------------
// helpers of the fp32 kernel
// ---------------------------------------------------------------------------
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

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
// output; D a multiple of 16 up to 256.
// ---------------------------------------------------------------------------
constexpr int kSimtThreads = 128;

struct SimtShared {
  float q[256][kSimtCols];            // [d][c]
  float pr[kTileKeys][kSimtCols];     // probabilities times the block's scale
  float red[4][kSimtCols];
  float m[kSimtCols], f[kSimtCols], l[kSimtCols];
  Segment seg;
  Group g;
};

// A page of the group: its rows in memory (NULL: none or a bad block id), its
// first key, its scale.
struct PageRef {
  const uint8_t *rows;
  float scale;
  long long key0;
  bool comp, there;
};
__device__ __forceinline__ PageRef page_ref(const AttnParams &p, const Pages &pg, int r, int v) {
  PageRef x;
  x.rows = nullptr;
  x.there = v < pg.nraw + pg.ncomp;
  x.comp = v >= pg.nraw;
  x.scale = __int_as_float(0x7fc00000);
  x.key0 = 0;
  if (!x.there) return x;
  const CacheSet &s = x.comp ? p.comp : p.raw;
  const int page = x.comp ? v - pg.nraw : pg.rp0 + v;
  x.key0 = (long long)page << p.log_bs;
  const int id = s.table[(size_t)r * s.cols + page % s.cols];
  if (id < 0 || id >= s.nblocks) return x;
  x.rows = s.pool + ((size_t)id << p.log_bs) * p.D;
  x.scale = s.scale[id];
  return x;
}

__global__ void __launch_bounds__(kSimtThreads) hca_cache_simt_kernel(const AttnParams p) {
  extern __shared__ uint8_t keys[];  // [128][D + 4] bytes: a row's words fall into different banks
  __shared__ SimtShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long ntiles = p.hdr->ntiles;
  if (ntiles < 0) {
    poison<float>(p);
    return;
  }
  const long long quota = cta_quota(ntiles, p.grid, kMinTiles);
  const long long c0 = quota * blockIdx.x, c1 = min(c0 + quota, ntiles);
  if (c0 >= c1) return;
  if (warp == 0) {
    const int g = find_group(p.groups, p.hdr->ngroups, c0);
    if (lane == 0) p.first[blockIdx.x] = g;
    if (lane == 0) sh.red[0][0] = __int_as_float(g);
  }
  __syncthreads();
  int gi = __float_as_int(sh.red[0][0]);
  const int pitch = p.D + 4;
  // output threads: dimension d, keys k0, k0 + kstep, ...
  int dpad = 16;
  while (dpad < p.D && dpad < kSimtThreads) dpad *= 2;
  const int kstep = kSimtThreads / dpad, kfirst = tid / dpad;
  for (long long at = c0; at < c1; ++gi) {
    __syncthreads();
    const Group g = p.groups[gi];
    const Segment seg = segment_of(g, c0, c1, blockIdx.x);
    at = g.tile0 + seg.j1;
    const int nreal = real_columns(p, g);
    const Pages pg = group_pages(g.pos0, g.npos, p.W, p.m, p.log_bs, p.comp.table != nullptr);
    const int h0 = g.slice * p.HS;
    for (int i = tid; i < p.D * kSimtCols; i += kSimtThreads) {
      const int c = i / p.D, d = i % p.D;
      float v = 0.f;
      if (c < nreal) v = static_cast<const float *>(p.q)[((size_t)(g.row0 + c / p.HS) * p.H + h0 + c % p.HS) * p.D + d];
      sh.q[d][c] = v;
    }
    if (tid < kSimtCols) {
      sh.m[tid] = -INFINITY;
      sh.l[tid] = 0.f;
    }
    float o[2][kSimtCols];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int c = 0; c < kSimtCols; ++c) o[x][c] = 0.f;
    const float sl2 = p.scale * 1.4426950408889634f;
    for (int j = seg.j0; j < seg.j1; ++j) {
      __syncthreads();
      // stage the tile's rows
      const int upr = p.D / 4;
      const int ppt = kTileKeys >> p.log_bs;
      for (int i = tid; i < kTileKeys * upr; i += kSimtThreads) {
        const int row = i / upr, u = i % upr;
        const PageRef x = page_ref(p, pg, g.r, j * ppt + (row >> p.log_bs));
        uint32_t w = 0;
        if (x.rows) w = reinterpret_cast<const uint32_t *>(x.rows + (size_t)(row & ((1 << p.log_bs) - 1)) * p.D)[u];
        *reinterpret_cast<uint32_t *>(keys + row * pitch + 4 * u) = w;
      }
      const PageRef x = page_ref(p, pg, g.r, j * ppt + (tid >> p.log_bs));
      int ca = 0, cb = 0;
      if (x.there) key_columns(x.comp, x.key0 + (tid & ((1 << p.log_bs) - 1)), g.pos0, g.npos, p.HS, p.W, p.m, ca, cb);
      const float sk = x.scale;
      if (!x.rows && x.there && cb > ca) p.hdr->status = HCA_ERR_CACHE;
      __syncthreads();
      float s[kSimtCols];
#pragma unroll
      for (int c = 0; c < kSimtCols; ++c) s[c] = 0.f;
      for (int u = 0; u < upr; ++u) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(keys + tid * pitch + 4 * u);
        const float2 a = f32x2_from_e4m3x2(w & 0xffffu), b = f32x2_from_e4m3x2(w >> 16);
        const float kk[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int c = 0; c < kSimtCols; ++c) s[c] = fmaf(kk[e], sh.q[4 * u + e][c], s[c]);
      }
#pragma unroll
      for (int c = 0; c < kSimtCols; ++c) {
        // a masked key's row may hold anything, NaN among it
        s[c] = c >= ca && c < cb ? s[c] * (sl2 * sk) : -INFINITY;
        float mx = s[c];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        if (lane == 0) sh.red[warp][c] = mx;
      }
      __syncthreads();
      if (tid < kSimtCols) {
        const float mx = fmaxf(fmaxf(sh.red[0][tid], sh.red[1][tid]), fmaxf(sh.red[2][tid], sh.red[3][tid]));
        const float mo = sh.m[tid], mn = fmaxf(mo, mx);
        sh.f[tid] = mn == -INFINITY ? 1.f : exp2f(mo - mn);
        sh.m[tid] = mn;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kSimtCols; ++c) {
        const float mn = sh.m[c];
        const float e = s[c] == -INFINITY ? 0.f : exp2f(s[c] - mn);
        sh.pr[tid][c] = e == 0.f ? 0.f : e * sk;
        float sum = e;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
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
      if (tid < kSimtCols)
        sh.l[tid] = sh.l[tid] * sh.f[tid] + ((sh.red[0][tid] + sh.red[1][tid]) + (sh.red[2][tid] + sh.red[3][tid]));
      for (int x2 = 0; x2 < 2; ++x2) {
        const int d = tid % dpad + x2 * kSimtThreads;
        if (d >= p.D) break;
        float acc[kSimtCols];
#pragma unroll
        for (int c = 0; c < kSimtCols; ++c) acc[c] = 0.f;
        for (int k = kfirst; k < kTileKeys; k += kstep) {
          const float v = f32x2_from_e4m3x2(keys[k * pitch + d]).x;
#pragma unroll
          for (int c = 0; c < kSimtCols; ++c) acc[c] = fmaf(sh.pr[k][c], v, acc[c]);
        }
#pragma unroll
        for (int c = 0; c < kSimtCols; ++c) {
          if (x2 == 0) o[0][c] = fmaf(o[0][c], sh.f[c], acc[c]);
          else o[1][c] = fmaf(o[1][c], sh.f[c], acc[c]);
        }
      }
    }
    __syncthreads();
    // join the key subsets of a dimension (D < 128), then write
    float *join = &sh.pr[0][0];  // [kstep][dpad][16] = 128 * 16
    if (kstep > 1) {
#pragma unroll
      for (int c = 0; c < kSimtCols; ++c) join[tid * kSimtCols + c] = o[0][c];
      __syncthreads();
      if (kfirst == 0)
        for (int k = 1; k < kstep; ++k)
#pragma unroll
          for (int c = 0; c < kSimtCols; ++c) o[0][c] += join[(k * dpad + tid) * kSimtCols + c];
    }
#pragma unroll
    for (int x2 = 0; x2 < 2; ++x2) {
      const int d = tid % dpad + x2 * kSimtThreads;
      if (d >= p.D || (kstep > 1 && kfirst > 0)) continue;
#pragma unroll
      for (int c = 0; c < kSimtCols; ++c) {
        if (c >= nreal) continue;
        if (seg.whole)
          static_cast<float *>(p.out)[((size_t)(g.row0 + c / p.HS) * p.H + h0 + c % p.HS) * p.D + d] = o[x2][c] / sh.l[c];
        else
          p.part_o[((size_t)seg.slot * kSimtCols + c) * p.D + d] = o[x2][c];
      }
    }
    if (tid < nreal) {
      if (seg.whole)
        p.lse[(size_t)(g.row0 + tid / p.HS) * p.H + h0 + tid % p.HS] = (sh.m[tid] + log2f(sh.l[tid])) * 0.69314718055994531f;
      else
        p.part_ml[(size_t)seg.slot * kSimtCols + tid] = make_float2(sh.m[tid], sh.l[tid]);
    }
  }
}

// ---------------------------------------------------------------------------
// combine: out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i over a group's parts
// ---------------------------------------------------------------------------
constexpr int kCombineWarps = 4;

// Block (c, y): the group that crosses the border between CTAs c and c + 1 and
// no earlier border; columns y, y + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(32 * kCombineWarps) hca_cache_combine_kernel(const AttnParams p) {
  __shared__ float4 acc[kCombineWarps][64];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long ntiles = p.hdr->ntiles;
  if (ntiles <= 0) return;
  if (p.hdr->status == HCA_ERR_TIMEOUT) {
    poison<T>(p);
    return;
  }
  const long long quota = cta_quota(ntiles, p.grid, kMinTiles);
  const long long border = quota * (blockIdx.x + 1);
  if (border >= ntiles) return;
  const Group g = p.groups[p.first[blockIdx.x + 1]];
  if (g.tile0 >= border || g.tile0 < border - quota) return;  // does not cross, or crosses an earlier border
  const int cta0 = blockIdx.x;
  const int n = (int)((g.tile0 + g.ntiles - 1) / quota) - cta0 + 1;
  // the first part's slot is 0 only where the group begins with its CTA's range
  auto slot = [&](int i) { return (size_t)(2 * (cta0 + i) + (i == 0 && g.tile0 != quota * cta0 ? 1 : 0)); };
  const int nreal = real_columns(p, g), h0 = g.slice * p.HS;
  const int v4 = p.D / 4;  // float4 of a row, at most 64
  for (int c = blockIdx.y; c < nreal; c += gridDim.y) {
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, p.part_ml[slot(i) * p.NQ + c].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    for (int i = lane; i < n; i += 32) {
      const float2 ml = p.part_ml[slot(i) * p.NQ + c];
      if (ml.y != 0.f) L += exp2f(ml.x - M) * ml.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float4 s[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int i = warp; i < n; i += kCombineWarps) {
      const float2 ml = p.part_ml[slot(i) * p.NQ + c];
      const float w = ml.y == 0.f ? 0.f : exp2f(ml.x - M);
      const float4 *o = reinterpret_cast<const float4 *>(p.part_o + (slot(i) * p.NQ + c) * p.D);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (lane + 32 * x < v4 && w != 0.f) {
          const float4 v = o[lane + 32 * x];
          s[x].x = fmaf(w, v.x, s[x].x); s[x].y = fmaf(w, v.y, s[x].y);
          s[x].z = fmaf(w, v.z, s[x].z); s[x].w = fmaf(w, v.w, s[x].w);
        }
      }
    }
    __syncthreads();
    acc[warp][lane] = s[0];
    acc[warp][32 + lane] = s[1];
    __syncthreads();
    const size_t row = (size_t)(g.row0 + c / p.HS) * p.H + h0 + c % p.HS;
    if (tid < v4) {
      float4 t = acc[0][tid];
#pragma unroll
      for (int w = 1; w < kCombineWarps; ++w) {
        const float4 u = acc[w][tid];
        t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
      }
      const float inv = 1.f / L;
      T *o = static_cast<T *>(p.out) + row * p.D + 4 * tid;
      put(o, t.x * inv); put(o + 1, t.y * inv); put(o + 2, t.z * inv); put(o + 3, t.w * inv);
    }
    if (tid == 0) p.lse[row] = (M + log2f(L)) * 0.69314718055994531f;
  }
}

// Columns of a group for H heads: enough for one position's slice of heads, and
// for as many positions as the average request brings.  More columns share a
// key tile between more rows; unused ones cost tensor and exponential work.
bool on_tensor_cores(int dtype) { return dtype == HCA_BF16; }

int pick_columns(int N, int R, int H, int dtype) {
  if (!on_tensor_cores(dtype)) return kSimtCols;
  const int slices = (H + 127) / 128, HS = (H + slices - 1) / slices;
  const int T = R > 0 ? (N + R - 1) / R : 1;
  const long long want = (long long)HS * T;
  return want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 ? 64 : 128;
}

struct Layout {
  int NQ, HS, slices, P;
  size_t gmax;
  size_t off_gbase, off_groups, off_first, off_ml, off_o, bytes;
};

Layout layout_of(int N, int R, int H, int D, int dtype) {
  Layout l;
  l.NQ = pick_columns(N, R, H, dtype);
  const int most = on_tensor_cores(dtype) ? 128 : kSimtCols;
  l.slices = (H + most - 1) / most;
  l.HS = (H + l.slices - 1) / l.slices;
  l.P = l.slices == 1 ? l.NQ / l.HS : 1;
  l.gmax = ((size_t)N / l.P + R) * l.slices;
  const size_t slots = 2 * (size_t)max_ctas(l.NQ, on_tensor_cores(dtype));
  size_t at = kHeaderBytes;
  l.off_gbase = at;
  at += align_up(((size_t)R + 1) * sizeof(int32_t));
  l.off_groups = at;
  at += align_up(l.gmax * sizeof(Group));
  l.off_first = at;
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

cudaError_t cache_attn(const CacheAttnArgs &a, cudaStream_t st) {
  const Layout l = layout_of(a.N, a.R, a.H, a.D, a.dtype);
  char *ws = static_cast<char *>(a.ws);
  AttnParams p;
  p.q = a.q; p.start = a.start; p.held = a.held; p.raw = a.raw; p.comp = a.comp; p.out = a.out; p.lse = a.lse;
  p.hdr = reinterpret_cast<SchedHeader *>(ws);
  p.gbase = reinterpret_cast<int32_t *>(ws + l.off_gbase);
  p.groups = reinterpret_cast<Group *>(ws + l.off_groups);
  p.first = reinterpret_cast<int32_t *>(ws + l.off_first);
  p.part_ml = reinterpret_cast<float2 *>(ws + l.off_ml);
  p.part_o = reinterpret_cast<float *>(ws + l.off_o);
  p.N = a.N; p.R = a.R; p.H = a.H; p.D = a.D; p.W = a.W; p.m = a.m; p.log_bs = log2_int(a.bs);
  p.HS = l.HS; p.slices = l.slices; p.P = l.P; p.NQ = l.NQ;
  p.scale = a.scale; p.wait_ns = a.wait_ns; p.stall = a.stall;
  const int sms = tc::sm_count();
  if (sms <= 0) return cudaErrorNoDevice;
  const bool tcs = on_tensor_cores(a.dtype);
  p.grid = std::min((tcs ? tc_cache_ctas(l.NQ) : 4) * sms, max_ctas(l.NQ, tcs));
  {
    ProfScope prof(kKCacheSched, st);
    hca_cache_sched_kernel<<<1, kSchedThreads, 0, st>>>(p);
  }
  if (tcs) {
    const cudaError_t e = tc_cache_attn(p, st);
    if (e != cudaSuccess) return e;
  } else {
    static tc::SmemAttrOnce attr;
    const cudaError_t e = attr.ensure(reinterpret_cast<const void *>(hca_cache_simt_kernel), kTileKeys * (256 + 4));
    if (e != cudaSuccess) return e;
    ProfScope prof(kKCacheSimt, st);
    hca_cache_simt_kernel<<<p.grid, kSimtThreads, kTileKeys * (a.D + 4), st>>>(p);
  }
  {
    ProfScope prof(kKCacheCombine, st);
    const dim3 grid(p.grid - 1, min(p.NQ, 8));
    if (a.dtype == HCA_F32) hca_cache_combine_kernel<float><<<grid, 32 * kCombineWarps, 0, st>>>(p);
    else hca_cache_combine_kernel<__nv_bfloat16><<<grid, 32 * kCombineWarps, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace hca
