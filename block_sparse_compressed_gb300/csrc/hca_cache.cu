// hca_cache.cu -- serving: block tables and slot maps from request lengths
// (hca_cache_plan), and rows into the 8-bit cache (hca_cache_append).
//
// Plan.  With E(L) = floor(L / m) entries for L tokens, request r adds entries
// [E(held), E(held + added)).  Entry e lies in table column (e / bs) mod cols
// at row e mod bs; the blocks of columns that were empty come from the end of
// the free list, in the order of the requests.  Two exclusive sums over the
// requests (entries, blocks) say everything: one CTA computes them, and every
// slot and every new table entry follows from a search in them and the free list
// alone, so they are written in any order, by that CTA for a decode step or by
// one CTA for 1,024 of them for prompts (1,060,000 slots: 10.5 us on the GPU, 191
// with one CTA).  A few hundred integers in, one integer out for each entry:
// bound by the latency of a launch and a few dependent loads (6.4 us for 64
// requests' next tokens; the bytes are 0.6 us for the prompts).
//
// Append.  A run is a maximal stretch of rows with consecutive slots in one
// block.  Its block's scale s is a power of two, so an e4m3 value never changes
// when s is divided out and bringing a block's earlier rows to a larger scale
// rounds only what falls below the smallest normal e4m3.  Rows of one run are
// contiguous in x and in the pool, so a run is one flat conversion of n * D
// values after one maximum over them.  64,258 rows of 128 bf16 values take 10.3
// us, 2.4 TB/s: one wave of CTAs that each wait for slots, values and owners in
// turn, behind a kernel of the owners (500,000 rows: 43 us, 4.5 TB/s); 64 single
// rows take 5 us, latency.
#include <cuda_bf16.h>

#include <algorithm>

#include "hca_cache.cuh"
#include "tc_ptx.cuh"

namespace hca {
using namespace cache;

namespace {

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
// Slots that the planning CTA itself writes: 3,000 and 5,000 take it 8.3 and 10.4 us,
// a second kernel 8.3 for both (10,000: 12.5 and 8.3).
constexpr int kPlanOneCta = 4096;

struct PlanItem {
  long long entries;
  int e0, n0, n1;  // entries held; blocks held before and after
  int ok;
};

__device__ __forceinline__ PlanItem plan_item(const CachePlanArgs &a, int r) {
  PlanItem t = {0, 0, 0, 0, 1};
  if (r >= a.R) return t;
  const long long h = a.held[r], d = a.added[r];
  if (h < 0 || d < 0 || h + d > kMaxPos) {
    t.ok = 0;
    return t;
  }
  const int e1 = (int)(h + d) / a.m;
  t.e0 = (int)h / a.m;
  t.entries = e1 - t.e0;
  t.n0 = min((t.e0 + a.bs - 1) >> a.log_bs, a.cols);
  t.n1 = min((e1 + a.bs - 1) >> a.log_bs, a.cols);
  return t;
}

// Largest r with before[r] <= i, of r in [lo, hi).
__device__ __forceinline__ int find_request(const int32_t *before, int lo, int hi, int i) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// Up to kPlanThreads requests' sums and items in shared memory, where a slot's
// request is searched and looked up.
struct PlanNear {
  int32_t start[kPlanThreads + 1], taken[kPlanThreads + 1];
  int32_t e0[kPlanThreads], last[kPlanThreads], n0[kPlanThreads];  // first and last new entry, blocks held before
  __device__ __forceinline__ void put(int r, const PlanItem &t) {
    e0[r] = t.e0;
    last[r] = t.e0 + (int)t.entries - 1;
    n0[r] = t.n0;
  }
};

// Part `part` of `parts` of the slots and of the new table entries, by the
// threads of this block.  start, taken [R + 1]: entries and blocks in front of
// each request (near's, if it is given); avail: free blocks before the plan.
__device__ __forceinline__ void plan_fill(const CachePlanArgs &a, const int32_t *start, const int32_t *taken,
                                          const PlanNear *near, int avail, int part, int parts) {
  const int total = start[a.R], blocks = taken[a.R];
  const int per = (a.nslots + parts - 1) / parts, i0 = part * per, i1 = min(i0 + per, a.nslots);
  if (i0 < i1) {
    // the requests of this part
    const int r0 = i0 < total ? find_request(start, 0, a.R, i0) : 0;
    const int r1 = i0 < total ? find_request(start, r0, a.R, min(i1, total) - 1) + 1 : 0;
#pragma unroll 4
    for (int i = i0 + threadIdx.x; i < i1; i += blockDim.x) {
      int slot = -1;
      if (i < total) {
        const int r = find_request(start, r0, r1, i);
        int e0, last, n0;
        if (near) {
          e0 = near->e0[r];
          last = near->last[r];
          n0 = near->n0[r];
        } else {
          const PlanItem t = plan_item(a, r);
          e0 = t.e0;
          last = t.e0 + (int)t.entries - 1;
          n0 = t.n0;
        }
        const int e = e0 + i - start[r], page = e >> a.log_bs;
        if ((last >> a.log_bs) - page < a.cols) {  // else a later new entry takes the row
          const int col = page < a.cols ? page : page % a.cols;
          const int id = col < n0 ? a.table[(size_t)r * a.cols + col] : a.free_blocks[avail - 1 - taken[r] - (col - n0)];
          if (id >= 0 && id < a.nblocks) slot = (id << a.log_bs) + (e & (a.bs - 1));
          else atomicExch(a.status, HCA_ERR_CACHE);
        }
      }
      a.slots[i] = slot;
    }
  }
  const int bper = (blocks + parts - 1) / parts, k1 = min((part + 1) * bper, blocks);
  for (int k = part * bper + threadIdx.x; k < k1; k += blockDim.x) {
    const int r = find_request(taken, 0, a.R, k), n0 = near ? near->n0[r] : plan_item(a, r).n0;
    a.table[(size_t)r * a.cols + n0 + k - taken[r]] = a.free_blocks[avail - 1 - k];
  }
}

__global__ void __launch_bounds__(kPlanThreads) hca_cache_plan_kernel(const CachePlanArgs a) {
  __shared__ long long tmp[33];
  __shared__ PlanNear near;
  const int tid = threadIdx.x;
  tc::pdl_launch_dependents();  // the fill kernel waits for this one's end by itself
  const int avail = *a.free_in;
  const int nt = blockDim.x;
  const bool few = a.R <= nt;
  // totals first: a plan that does not fit changes nothing
  long long entries = 0, blocks = 0;
  bool ok = avail >= 0 && avail <= a.nfree;
  PlanItem t = {0, 0, 0, 0, 1};
  for (int r = tid; r < a.R; r += nt) {
    t = plan_item(a, r);
    ok = ok && t.ok;
    entries += t.entries;
    blocks += t.n1 - t.n0;
  }
  long long all_entries, all_blocks;
  long long s = block_scan(entries, tmp, all_entries), k = block_scan(blocks, tmp, all_blocks);
  const bool valid = __syncthreads_and(ok);
  const bool go = valid && all_entries <= a.nslots && all_blocks <= avail;
  if (tid == 0) {
    *a.status = go ? HCA_OK : valid ? HCA_ERR_CAPACITY : HCA_ERR_CACHE;
    *a.free_out = go ? avail - (int)all_blocks : avail;
    *a.avail = avail;
    a.start[a.R] = near.start[few ? a.R : 0] = go ? (int)all_entries : 0;
    a.taken[a.R] = near.taken[few ? a.R : 0] = go ? (int)all_blocks : 0;
  }
  if (few) {
    // one request a thread: its sums are at hand
    if (tid < a.R) {
      a.start[tid] = near.start[tid] = go ? (int)s : 0;
      a.taken[tid] = near.taken[tid] = go ? (int)k : 0;
      near.put(tid, t);
    }
  } else {
    long long at = 0, took = 0;
    for (int r0 = 0; r0 < a.R; r0 += nt) {
      const int r = r0 + tid;
      PlanItem x = {0, 0, 0, 0, 1};
      if (go) x = plan_item(a, r);
      long long n, nb;
      s = at + block_scan(x.entries, tmp, n);
      k = took + block_scan(x.n1 - x.n0, tmp, nb);
      if (r < a.R) {
        a.start[r] = (int)s;
        a.taken[r] = (int)k;
      }
      at += n;
      took += nb;
    }
  }
  __syncthreads();
  if (a.nslots <= kPlanOneCta) plan_fill(a, few ? near.start : a.start, few ? near.taken : a.taken, few ? &near : nullptr, avail, 0, 1);
}

// Slots of a CTA (198,600 and 1,059,918 slots: 10.4 and 10.3 us; 512 of them 8.4 and
// 12.4, 2,048 12.5 and 10.3).
constexpr int kFillThreads = 256, kSlotsPerCta = 1024;

__global__ void __launch_bounds__(kFillThreads) hca_cache_fill_kernel(const CachePlanArgs a) {
  __shared__ PlanNear near;
  const bool few = a.R <= kPlanThreads;
  if (few)
    for (int r = threadIdx.x; r < a.R; r += kFillThreads) near.put(r, plan_item(a, r));
  tc::pdl_wait();
  const int avail = *a.avail;
  if (few) {
#pragma unroll 4
    for (int r = threadIdx.x; r <= a.R; r += kFillThreads) {
      near.start[r] = a.start[r];
      near.taken[r] = a.taken[r];
    }
    __syncthreads();
  }
  plan_fill(a, few ? near.start : a.start, few ? near.taken : a.taken, few ? &near : nullptr, avail, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// Up to this many rows (a decode step's) one cluster of CTAs does it all: a run
// looks through all slots for others of its block.  For more the blocks are
// claimed by a kernel in front (measured: 2 us more for 64 rows).
constexpr int kAppendLook = 256;
constexpr int kSmallCtas = 8, kSmallThreads = 512, kSmallWarps = kSmallCtas * kSmallThreads / 32;

// Row t begins a run: its slot is not the one behind row t - 1's, or it is the
// first of a block.
__device__ __forceinline__ bool begins_run(const CacheAppendArgs &a, int t) {
  const int s = a.slots[t];
  if (s < 0 || s >= a.nblocks * a.bs) return false;
  return t == 0 || (s & (a.bs - 1)) == 0 || a.slots[t - 1] != s - 1;
}

// Every run writes its first row's index into its block's owner word.  A run
// that finds another's there (rows of one block that are not adjacent in x, or
// a slot twice) is reported and left out: it would race with the other.
__global__ void hca_cache_claim_kernel(const CacheAppendArgs a) {
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  tc::pdl_launch_dependents();  // the rows' kernel waits for this one's end by itself
  if (t == 0) *a.status = HCA_OK;
  if (t < a.N && begins_run(a, t)) a.owner[a.slots[t] >> a.log_bs] = t;
}

// 16 values as they lie in memory
template <typename T>
struct Held {
  uint4 w[sizeof(T)];
};

template <typename T>
__device__ __forceinline__ void hold16(const T *p, Held<T> &h) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) h.w[i] = reinterpret_cast<const uint4 *>(p)[i];
}

template <typename T>
__device__ __forceinline__ void expand16(const Held<T> &h, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) {
    const uint32_t w[4] = {h.w[i].x, h.w[i].y, h.w[i].z, h.w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(T) == 4) {
        v[4 * i + k] = __uint_as_float(w[k]);
      } else {
        v[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
        v[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&v)[16]) {
  Held<T> h;
  hold16(p, h);
  expand16(h, v);
}

__device__ __forceinline__ uint4 pack16(const float (&v)[16]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = e4m3x2(v[4 * i], v[4 * i + 1]) | (e4m3x2(v[4 * i + 2], v[4 * i + 3]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest magnitude of the finite ones.
__device__ __forceinline__ float finite_max(const float (&v)[16]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float f = fabsf(v[i]);
    if (f < INFINITY) m = fmaxf(m, f);
  }
  return m;
}

__device__ __forceinline__ uint4 quantise16(float (&v)[16], float inv) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = fmaf(v[i], 0.f, v[i] * inv);  // an infinity becomes NaN, not 448
  return pack16(v);
}

// The scale of block blk with new values up to amax from row off on; the rows in
// front of them are brought to it by `nthreads` threads.
__device__ __forceinline__ float settle_scale(const CacheAppendArgs &a, int blk, int off, float amax, int tid, int nthreads,
                                              int &err) {
  const float s = exp2_int(scale_exponent(amax));
  if (off == 0) return s;
  const float old = a.scale[blk];
  if (!(old > 0.f && old < INFINITY)) {
    err = HCA_ERR_CACHE;
    return s;
  }
  if (old >= s) return old;
  const float f = old / s;
  uint4 *rows = reinterpret_cast<uint4 *>(a.pool + (size_t)blk * a.bs * a.D);
  for (int u = tid; u < off * a.D / 16; u += nthreads) {
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
  return s;
}

// The run that begins at row t, by one warp; returns an error status.
template <typename T, bool kClaimed>
__device__ __forceinline__ int append_run(const CacheAppendArgs &a, int t, int lane) {
  const int slot = a.slots[t];
  const int blk = slot >> a.log_bs, off = slot & (a.bs - 1);
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
  int err = HCA_OK;
  if constexpr (kClaimed) {
    if (a.owner[blk] != t) return HCA_ERR_CACHE;
  } else {
    // another run of the block: the first one of them all is written
    bool before = false, behind = false;
    for (int u = lane; u < a.N; u += 32) {
      const bool same = a.slots[u] >> a.log_bs == blk;
      before = before || (same && u < t);
      behind = behind || (same && u >= t + n);
    }
    if (__any_sync(0xffffffffu, before || behind)) err = HCA_ERR_CACHE;
    if (__any_sync(0xffffffffu, before)) return err;
  }
  const T *x = static_cast<const T *>(a.x) + (size_t)t * a.D;
  uint8_t *dst = a.pool + (size_t)slot * a.D;
  const int units = n * a.D / 16;
  float amax = 0.f;
#pragma unroll 4
  for (int u = lane; u < units; u += 32) {
    float v[16];
    load16(x + (size_t)u * 16, v);
    amax = fmaxf(amax, finite_max(v));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = settle_scale(a, blk, off, amax, lane, 32, err);
  __syncwarp();
  if (lane == 0) a.scale[blk] = s;
  const float inv = 1.f / s;
#pragma unroll 4
  for (int u = lane; u < units; u += 32) {
    float v[16];
    load16(x + (size_t)u * 16, v);
    *reinterpret_cast<uint4 *>(dst + (size_t)u * 16) = quantise16(v, inv);
  }
  return err;
}

// A CTA takes the runs that begin in `rows` consecutive rows: long ones all
// threads together, so that a block's rows are in flight at once, short ones a
// warp each.  Values wait for their block's scale as they came: as fp32 they took
// 96 registers, 5 CTAs an SM and 12.3 us where it is 8 and 10.3 now.  Long is from
// kLongRun rows on: 1,500 runs of 1 to 12 rows take 8.4 us, 10.3 from 4 on; 8 runs
// of up to 300 rows 6.2, 7.4 from 16 on (which is better for blocks of 16: 64,258
// rows 12.6 for 13.0).
constexpr int kChunkThreads = 128, kChunkRows = 64, kLongRun = 8;
constexpr int kWindow = kChunkRows + 128;  // rows looked at: the last run may go on for a block

template <typename T>
__global__ void __launch_bounds__(kChunkThreads, sizeof(T) == 2 ? 8 : 5) hca_cache_append_kernel(const CacheAppendArgs a, int rows) {
  __shared__ int slot_of[kWindow + 1];       // slots of rows t0 - 1, t0, ...
  __shared__ uint32_t breaks[kWindow / 32];  // rows that are not behind the one in front
  __shared__ int lead[kChunkRows], nlead;
  __shared__ float red[kChunkThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * rows, cnt = min(rows, a.N - t0), limit = a.nblocks * a.bs;
  for (int i = tid; i <= kWindow; i += kChunkThreads) {
    const int t = t0 - 1 + i;
    slot_of[i] = t >= 0 && t < a.N ? a.slots[t] : -2;
  }
  if (tid == 0) nlead = 0;
  __syncthreads();
  int err = HCA_OK;
  for (int i = tid; i < kWindow; i += kChunkThreads) {
    const int s = slot_of[i + 1];
    const bool brk = s < 0 || (s & (a.bs - 1)) == 0 || slot_of[i] != s - 1;
    const uint32_t b = __ballot_sync(0xffffffffu, brk);
    if (lane == 0) breaks[i >> 5] = b;
    if (i < cnt && s >= limit) err = HCA_ERR_CACHE;
    // the order of the list does not matter
    if (i < cnt && brk && s >= 0 && s < limit) lead[atomicAdd(&nlead, 1)] = i;
  }
  __syncthreads();
  auto length = [&](int i) {
    int w = (i + 1) >> 5;
    uint32_t b = w < kWindow / 32 ? breaks[w] & (0xffffffffu << ((i + 1) & 31)) : 0;
    while (!b && ++w < kWindow / 32) b = breaks[w];
    return (b ? 32 * w + __ffs(b) - 1 : kWindow) - i;
  };
  for (int j = 0; j < nlead; ++j) {
    const int i = lead[j], n = length(i);
    if (n < kLongRun) continue;
    const int t = t0 + i, slot = slot_of[i + 1], blk = slot >> a.log_bs, off = slot & (a.bs - 1);
    const T *x = static_cast<const T *>(a.x) + (size_t)t * a.D;
    uint8_t *dst = a.pool + (size_t)slot * a.D;
    const int units = n * a.D / 16;
    constexpr int kHold = 4;  // units of 16 values that a thread keeps
    Held<T> held[kHold];
    float v[16], amax = 0.f;
    for (int u0 = 0; u0 < units; u0 += kHold * kChunkThreads) {
#pragma unroll
      for (int k = 0; k < kHold; ++k) {
        const int u = u0 + k * kChunkThreads + tid;
        if (u < units) hold16(x + (size_t)u * 16, held[k]);
      }
#pragma unroll
      for (int k = 0; k < kHold; ++k)
        if (u0 + k * kChunkThreads + tid < units) {
          expand16(held[k], v);
          amax = fmaxf(amax, finite_max(v));
        }
    }
    tc::pdl_wait();  // for the owners
    if (a.owner[blk] != t) {
      err = HCA_ERR_CACHE;
      continue;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    __syncthreads();
    if (lane == 0) red[warp] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float s = settle_scale(a, blk, off, amax, tid, kChunkThreads, err);
    __syncthreads();  // every thread has read the old scale
    if (tid == 0) a.scale[blk] = s;
    const float inv = 1.f / s;
    for (int u0 = 0; u0 < units; u0 += kHold * kChunkThreads) {
#pragma unroll
      for (int k = 0; k < kHold; ++k) {
        const int u = u0 + k * kChunkThreads + tid;
        if (u < units) {
          if (units > kHold * kChunkThreads) hold16(x + (size_t)u * 16, held[k]);  // else it is still there
          expand16(held[k], v);
          *reinterpret_cast<uint4 *>(dst + (size_t)u * 16) = quantise16(v, inv);
        }
      }
    }
  }
  tc::pdl_wait();
  for (int j = warp; j < nlead; j += kChunkThreads / 32)
    if (length(lead[j]) < kLongRun) err = max(err, append_run<T, true>(a, t0 + lead[j], lane));
  if (__any_sync(0xffffffffu, err != HCA_OK) && lane == 0) atomicExch(a.status, HCA_ERR_CACHE);
}

template <typename T, bool kClaimed>
__device__ __forceinline__ int append_row(const CacheAppendArgs &a, int t, int lane) {
  if (a.slots[t] >= a.nblocks * a.bs) return HCA_ERR_CACHE;
  return begins_run(a, t) ? append_run<T, kClaimed>(a, t, lane) : HCA_OK;
}

template <typename T>
__global__ void __cluster_dims__(kSmallCtas, 1, 1) __launch_bounds__(kSmallThreads)
    hca_cache_append_small_kernel(const CacheAppendArgs a) {
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = HCA_OK;
  int err = HCA_OK;
  for (int t = (threadIdx.x >> 5) * kSmallCtas + blockIdx.x; t < a.N; t += kSmallWarps)
    err = max(err, append_row<T, false>(a, t, lane));
  // the status has been reset before anybody raises it
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (err != HCA_OK && lane == 0) atomicExch(a.status, err);
}

}  // namespace

size_t cache_plan_ws_bytes(int R) { return kHeaderBytes + align_up(((size_t)R + 1) * sizeof(int32_t)); }

cudaError_t cache_plan(const CachePlanArgs &args, void *ws, cudaStream_t st) {
  CachePlanArgs a = args;
  a.status = static_cast<int32_t *>(ws);
  a.avail = a.status + 1;
  a.taken = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + kHeaderBytes);
  a.log_bs = 0;
  while ((1 << a.log_bs) < a.bs) ++a.log_bs;
  ProfScope prof(kKCachePlan, st);
  // a thread for each request, and for the slots that this CTA writes
  const int want = std::max(a.R, a.nslots <= kPlanOneCta ? a.nslots : 0);
  hca_cache_plan_kernel<<<1, std::min(std::max((want + 31) / 32 * 32, 32), kPlanThreads), 0, st>>>(a);
  if (a.nslots > kPlanOneCta)
    return launch_behind(hca_cache_fill_kernel, dim3((a.nslots + kSlotsPerCta - 1) / kSlotsPerCta), kFillThreads, 0, st, a);
  return cudaGetLastError();
}

cudaError_t cache_append(const CacheAppendArgs &args, cudaStream_t st) {
  CacheAppendArgs a = args;
  a.log_bs = 0;
  while ((1 << a.log_bs) < a.bs) ++a.log_bs;
  const bool f32 = a.dtype == HCA_F32;
  ProfScope prof(kKCacheAppend, st);
  if (a.N <= kAppendLook) {
    if (f32) hca_cache_append_small_kernel<float><<<kSmallCtas, kSmallThreads, 0, st>>>(a);
    else hca_cache_append_small_kernel<__nv_bfloat16><<<kSmallCtas, kSmallThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  hca_cache_claim_kernel<<<(a.N + 255) / 256, 256, 0, st>>>(a);
  // enough CTAs for every SM, but no more than one for each block of a long prompt
  // (64,258 rows in blocks of 64 and of 16, and 1,500 runs of 1 to 40 rows: 10.5, 13.0
  // and 12.2 us; N / 512 10.5, 14.5 and 14.6; N / 2048 11.3, 12.9 and 12.4)
  const int rows = std::min(std::max(a.N / 1024, 4), kChunkRows);
  const int grid = (a.N + rows - 1) / rows;
  return f32 ? launch_behind(hca_cache_append_kernel<float>, dim3(grid), kChunkThreads, 0, st, a, rows)
             : launch_behind(hca_cache_append_kernel<__nv_bfloat16>, dim3(grid), kChunkThreads, 0, st, a, rows);
}

}  // namespace hca
