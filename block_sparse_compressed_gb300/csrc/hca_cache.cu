// hca_cache.cu -- serving: block tables and slot maps from request lengths
// (hca_cache_plan), and rows into the 8-bit cache (hca_cache_append).
//
// Plan.  With E(L) = floor(L / m) entries for L tokens, request r adds entries
// [E(held), E(held + added)).  Entry e lies in table column (e / bs) mod cols
// at row e mod bs; the blocks of columns that were empty come from the end of
// the free list, in the order of the requests.  Two exclusive sums over the
// requests (entries, blocks) say everything: one CTA computes them, then the
// slots follow from a search in the first.  A few hundred integers in, one
// integer out for each entry: bound by latency for a decode step, by the slot
// writes for long prompts.
//
// Append.  A run is a maximal stretch of rows with consecutive slots in one
// block.  Its block's scale s is a power of two, so an e4m3 value never changes
// when s is divided out and bringing a block's earlier rows to a larger scale
// rounds only what falls below the smallest normal e4m3.  Rows of one run are
// contiguous in x and in the pool, so a run is one flat conversion of n * D
// values after one maximum over them.
#include <cuda_bf16.h>

#include "hca_cache.cuh"

namespace hca {
using namespace cache;

namespace {

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanOneCta = 4096;  // slots that the planning CTA itself writes

struct PlanItem {
  long long entries;
  int n0, n1;  // blocks held before and after
  int ok;
};

__device__ __forceinline__ PlanItem plan_item(const CachePlanArgs &a, int r) {
  PlanItem t = {0, 0, 0, 1};
  if (r >= a.R) return t;
  const long long h = a.held[r], d = a.added[r];
  if (h < 0 || d < 0 || h + d > kMaxPos) {
    t.ok = 0;
    return t;
  }
  const int e0 = (int)h / a.m, e1 = (int)(h + d) / a.m;
  t.entries = e1 - e0;
  t.n0 = min((e0 + a.bs - 1) / a.bs, a.cols);
  t.n1 = min((e1 + a.bs - 1) / a.bs, a.cols);
  return t;
}

// Slots [i0, i1) of the plan, by the threads of this block.
__device__ __forceinline__ void fill_slots(const CachePlanArgs &a, const int32_t *start, int i0, int i1) {
  const int total = start[a.R];
  for (int i = i0 + threadIdx.x; i < i1; i += blockDim.x) {
    int slot = -1;
    if (i < total) {
      int lo = 0, hi = a.R;  // start[lo] <= i < start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid; else hi = mid;
      }
      const int e0 = a.held[lo] / a.m, e1 = (a.held[lo] + a.added[lo]) / a.m;
      const int e = e0 + i - start[lo];
      const int page = e / a.bs;
      if ((e1 - 1) / a.bs - page < a.cols) {  // else a later new entry takes the row
        const int id = a.table[(size_t)lo * a.cols + page % a.cols];
        if (id >= 0 && id < a.nblocks) slot = id * a.bs + e % a.bs;
        else atomicExch(a.status, HCA_ERR_CACHE);
      }
    }
    a.slots[i] = slot;
  }
}

__global__ void __launch_bounds__(kPlanThreads) hca_cache_plan_kernel(const CachePlanArgs a) {
  __shared__ long long tmp[33];
  const int tid = threadIdx.x;
  const int avail = *a.free_in;
  // totals first: a plan that does not fit changes nothing
  long long entries = 0, blocks = 0;
  bool ok = avail >= 0 && avail <= a.nfree;
  for (int r = tid; r < a.R; r += kPlanThreads) {
    const PlanItem t = plan_item(a, r);
    ok = ok && t.ok;
    entries += t.entries;
    blocks += t.n1 - t.n0;
  }
  long long all_entries, all_blocks;
  block_scan(entries, tmp, all_entries);
  block_scan(blocks, tmp, all_blocks);
  const bool valid = __syncthreads_and(ok);
  const bool fits = all_entries <= a.nslots && all_blocks <= avail;
  if (tid == 0) *a.status = !valid ? HCA_ERR_CACHE : fits ? HCA_OK : HCA_ERR_CAPACITY;
  const bool go = valid && fits;
  long long at = 0, taken = 0;
  for (int r0 = 0; r0 < a.R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    PlanItem t = {0, 0, 0, 1};
    if (go) t = plan_item(a, r);
    long long n, nb;
    const long long s = at + block_scan(t.entries, tmp, n);
    const long long k0 = taken + block_scan(t.n1 - t.n0, tmp, nb);
    if (r < a.R) {
      a.start[r] = (int)s;
      for (int j = t.n0; j < t.n1; ++j) {
        const int id = a.free_blocks[avail - 1 - (int)k0 - (j - t.n0)];
        a.table[(size_t)r * a.cols + j] = id;
      }
    }
    at += n;
    taken += nb;
  }
  if (tid == 0) {
    a.start[a.R] = (int)at;
    *a.free_out = avail - (int)taken;
  }
  __syncthreads();
  if (a.nslots <= kPlanOneCta) fill_slots(a, a.start, 0, a.nslots);
}

constexpr int kSlotThreads = 256, kSlotsPerCta = 2048;

__global__ void __launch_bounds__(kSlotThreads) hca_cache_slots_kernel(const CachePlanArgs a) {
  const int i0 = blockIdx.x * kSlotsPerCta;
  fill_slots(a, a.start, i0, min(i0 + kSlotsPerCta, a.nslots));
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;
constexpr int kRowsPerCta = 8;

// Row t begins a run: its slot is not the one behind row t - 1's, or it is the
// first of a block.
__device__ __forceinline__ bool begins_run(const CacheAppendArgs &a, int t) {
  const int s = a.slots[t];
  if (s < 0 || s >= a.nblocks * a.bs) return false;
  return t == 0 || s % a.bs == 0 || a.slots[t - 1] != s - 1;
}

// Every run writes its first row's index into its block's owner word.  A run
// that finds another's there (rows of one block that are not adjacent in x, or
// a slot twice) is reported and left out: it would race with the other.
__global__ void hca_cache_claim_kernel(const CacheAppendArgs a) {
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t == 0) *a.status = HCA_OK;
  if (t < a.N && begins_run(a, t)) a.owner[a.slots[t] / a.bs] = t;
}

template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&v)[16]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = reinterpret_cast<const float4 *>(p)[i];
      v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = reinterpret_cast<const uint4 *>(p)[i];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
        v[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ uint4 pack16(const float (&v)[16]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = e4m3x2(v[4 * i], v[4 * i + 1]) | (e4m3x2(v[4 * i + 2], v[4 * i + 3]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One run by one warp.
template <typename T>
__device__ __forceinline__ void append_run(const CacheAppendArgs &a, int t, int lane) {
  const int slot = a.slots[t];
  const int blk = slot / a.bs, off = slot % a.bs;
  // length of the run: up to the block's end
  int n = 1;
  const int most = min(a.bs - off, a.N - t);
  for (int i0 = 1; i0 < most; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < most && a.slots[t + i] == slot + i;
    const uint32_t b = __ballot_sync(0xffffffffu, in);
    const int k = b == 0xffffffffu ? 32 : __ffs(~b) - 1;
    n += k;
    if (k < 32) break;
  }
  if (a.owner[blk] != t) {
    if (lane == 0) atomicExch(a.status, HCA_ERR_CACHE);
    return;
  }
  const T *x = static_cast<const T *>(a.x) + (size_t)t * a.D;
  uint8_t *dst = a.pool + (size_t)slot * a.D;
  const int units = n * a.D / 16;
  float amax = 0.f;
  for (int u = lane; u < units; u += 32) {
    float v[16];
    load16(x + (size_t)u * 16, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float f = fabsf(v[i]);
      if (f < INFINITY) amax = fmaxf(amax, f);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  float s = exp2_int(scale_exponent(amax));
  if (off > 0) {
    const float old = a.scale[blk];
    if (!(old > 0.f && old < INFINITY)) {
      if (lane == 0) atomicExch(a.status, HCA_ERR_CACHE);
    } else if (old < s) {
      // the block's earlier rows to the larger scale
      const float f = old / s;
      uint4 *rows = reinterpret_cast<uint4 *>(a.pool + (size_t)blk * a.bs * a.D);
      for (int u = lane; u < off * a.D / 16; u += 32) {
        const uint4 w = rows[u];
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 p = f32x2_from_e4m3x2((in[i >> 1] >> (16 * (i & 1))) & 0xffffu);
          v[2 * i] = p.x * f;
          v[2 * i + 1] = p.y * f;
        }
        rows[u] = pack16(v);
      }
    } else {
      s = old;
    }
  }
  __syncwarp();
  if (lane == 0) a.scale[blk] = s;
  const float inv = 1.f / s;
  for (int u = lane; u < units; u += 32) {
    float v[16];
    load16(x + (size_t)u * 16, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = fmaf(v[i], 0.f, v[i] * inv);  // an infinity becomes NaN, not 448
    *reinterpret_cast<uint4 *>(dst + (size_t)u * 16) = pack16(v);
  }
}

template <typename T>
__global__ void __launch_bounds__(kAppendThreads) hca_cache_append_kernel(const CacheAppendArgs a) {
  const int t = blockIdx.x * kRowsPerCta + (threadIdx.x >> 5);
  if (t >= a.N) return;
  const int lane = threadIdx.x & 31;
  const int s = a.slots[t];
  if (s >= a.nblocks * a.bs) {
    if (lane == 0) atomicExch(a.status, HCA_ERR_CACHE);
    return;
  }
  if (begins_run(a, t)) append_run<T>(a, t, lane);
}

}  // namespace

cudaError_t cache_plan(const CachePlanArgs &a, cudaStream_t st) {
  ProfScope prof(kKCachePlan, st);
  hca_cache_plan_kernel<<<1, kPlanThreads, 0, st>>>(a);
  if (a.nslots > kPlanOneCta)
    hca_cache_slots_kernel<<<(a.nslots + kSlotsPerCta - 1) / kSlotsPerCta, kSlotThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t cache_append(const CacheAppendArgs &a, cudaStream_t st) {
  ProfScope prof(kKCacheAppend, st);
  hca_cache_claim_kernel<<<(a.N + 255) / 256, 256, 0, st>>>(a);
  const int grid = (a.N + kRowsPerCta - 1) / kRowsPerCta;
  if (a.dtype == HCA_F32) hca_cache_append_kernel<float><<<grid, kAppendThreads, 0, st>>>(a);
  else hca_cache_append_kernel<__nv_bfloat16><<<grid, kAppendThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace hca
