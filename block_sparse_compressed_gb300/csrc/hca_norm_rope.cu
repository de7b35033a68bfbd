// hca_norm_rope.cu -- what stands between a layer's projections and its
// attention: the norm of each head's query and of the shared kv row, and the
// rotation of some of their columns by the token's position, in one pass over
// the rows; their backward; and the rotation alone (the attention's output is
// turned back by it, since kv is key and value at once).
//
//   r = (mean_d x_d^2 + eps)^-1/2,  y = x r w
//   theta_p = sum_a c_a f[a][p]     angle of pair p at coordinates c
//   (u, v) -> (u cos - v sin, u sin + v cos) for the two columns of a pair
// Backward for g = dL/d(output):
//   g' = g turned by -theta,  dw = sum over rows of g' x r,
//   h = g' w,  dx = r (h - x r^2 mean_d(h x))
//
// Angles.  A position of 10^6 times a frequency of 1 is 10^6 radians, of which
// fp32 keeps a sixteenth.  So a frequency becomes a 64-bit fraction of a turn
// per unit, F = f / 2pi * 2^64 mod 2^64 (exact to 2^-64 turns),
// and a phase is sum_a c_a F[a] in integers, where the wrap-around of 64 bits is
// the reduction to one turn: off by 2^-33 turns an axis at most for any 32-bit
// coordinates.  The two upper bits (rounded) are the quadrant, the rest is an eighth
// of a turn at most; cos and sin are right to 3 2^-24.
//
// A row belongs to L neighbouring lanes in chunks of 16 bytes, so it is read once,
// stays in registers between the sum of its squares and its output, and is written
// once.  A block takes a tile of tokens and a range of heads: the tile's cos and sin
// are made once in shared memory, then each lane keeps those of its own columns and
// token in registers, times the weights, for all of the block's heads.
//
// Bounds.  Long sequences are bound by memory: forward of B = 1, H = 64, S = 65,536,
// D = 128 in bf16 (2.18 GB) 323 us, 99% of the measured copy bandwidth, backward
// (3.27 GB) 485 us, 99%; H = 16 in fp32 168 and 249 us, 100%.  (With a row's loads in its registers: 422 and 671 us; fp32
// one by one instead of in pairs, and addresses by multiplication: 354 and 631.)
// Shorter ones are bound by the blocks' beginnings, 2 us from the first instruction
// to the first row: 2,571 prompt tokens (86 MB) 16 us; one token of 64 requests 4 us, of
// which 2 are the launch (calls in a graph, all of these).  Few heads are bound by instructions, since a
// token's cos and sin and a lane's factors are for few rows: one head and kv of 524,288
// tokens 225 us (540 MB, 80 us; a thousand instructions of a warp for two rows a lane).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "hca_cache.cuh"
#include "tc_tiles.cuh"

namespace hca {
namespace {

constexpr int kThreads = 256;
constexpr int kRequestsInSmem = 1024;
enum Mode { kRope = 0, kFwd = 1, kBwd = 2 };

struct Args {
  NormRopeTensor t[2];  // queries, kv (H = 0: none)
  const int32_t *pos, *start, *held;
  const float *freq;
  float *part;          // [grid][2][D] sums of dw (backward)
  int B, S, D, R, axes, first, rot;
  float sign, eps;
  uint32_t tiles;       // token tiles of all batch rows
  uint32_t per_row;     // of a batch row
  uint32_t inv_np;      // 2^32 / (rot / 2), rounded up
  int tile, log_tile;   // tokens of a tile, a power of two
  int splits, per;      // head ranges of a tile, heads (of q, then kv) of a range
};

// 16 bytes of a row (a chunk: 8 columns of bf16, 4 of fp32) as they are in memory, and
// as packed pairs of fp32 in slots.  With neighbours for pairs of a rotation the slots
// are columns (0, 2), (4, 6), (1, 3), (5, 7), or (0, 2), (1, 3), so that the two
// columns of a rotation lie in slots i and i ^ kSlots / 2, which costs bf16 nothing:
// its halves are taken apart in any case.
template <typename T, bool HALVES>
struct Vec {
  static constexpr int kCols = 16 / (int)sizeof(T), kSlots = kCols / 2;
  uint32_t w[4];

  static __device__ __forceinline__ constexpr int column(int slot, int e) {
    return HALVES ? 2 * slot + e : slot % (kSlots / 2) * 4 + 2 * e + slot / (kSlots / 2);
  }
  __device__ __forceinline__ void load(const uint4 &u) { w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w; }
  __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]); }
  // the same chunk of lane `from`
  __device__ __forceinline__ Vec of(int from) const {
    Vec r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = __shfl_sync(0xffffffffu, w[i], from);
    return r;
  }
  __device__ __forceinline__ uint32_t at(int c) const {
    if constexpr (sizeof(T) == 4) return w[c];
    else return c & 1 ? w[c >> 1] & 0xffff0000u : w[c >> 1] << 16;
  }
  __device__ __forceinline__ void get(uint64_t (&f)[kSlots]) const {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) f[i] = tc::f32x2(at(column(i, 0)), at(column(i, 1)));
  }
  __device__ __forceinline__ void put(const uint64_t (&f)[kSlots]) {
    float v[kCols];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) tc::f32x2_split(f[i], v[column(i, 0)], v[column(i, 1)]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
      else w[i] = tc::pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
  }
};

__device__ __forceinline__ uint64_t pair(float a, float b) { return tc::f32x2(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float total(uint64_t v) {
  float a, b;
  tc::f32x2_split(v, a, b);
  return a + b;
}

// f / 2pi of a turn per unit as a 64-bit fraction: f = m 2^e times 2^128 / 2pi,
// whose bits from 64 - e on are the ones wanted.  (In doubles, which this GPU is slow
// at, a block's table took 1 us.)
__device__ __forceinline__ unsigned long long turns(float f) {
  constexpr uint32_t kInv2Pi[4] = {0x7d4d3770u, 0x7f09d5f4u, 0x9391054au, 0x28be60dbu};
  const uint32_t u = __float_as_uint(f), ex = (u >> 23) & 255;
  const uint32_t m = (u & 0x7fffffu) | (ex ? 0x800000u : 0u);
  uint32_t w[7] = {0, 0, 0, 0, 0, 0, 0};
  unsigned long long carry = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    carry += (unsigned long long)m * kInv2Pi[i];
    w[i] = (uint32_t)carry;
    carry >>= 32;
  }
  w[4] = (uint32_t)carry;
  const int shift = 64 - (max((int)ex, 1) - 150);  // 55 and more for f below 2^32
  uint32_t lo = 0, mid = 0, hi = 0;                // the three words that the 64 bits lie in
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    if (shift >> 5 == i) lo = w[i], mid = w[i + 1], hi = w[i + 2];
  }
  const unsigned long long t = (unsigned long long)__funnelshift_r(mid, hi, shift & 31) << 32 | __funnelshift_r(lo, mid, shift & 31);
  return u >> 31 ? 0ull - t : t;
}

// A frequency without an angle: of 2^64 and more, whose bits behind the point are not
// among the 128 above, an infinity or NaN.  With one all columns that turn are NaN.  (What
// looks for it takes 0.17 us: one token of 64 requests 3.77 to 3.94 in a graph.)
__device__ __forceinline__ int no_angle(float f) { return __float_as_uint(f) << 1 >= 191u << 24; }

// The rest of a phase, an eighth of a turn at most, in radians: the Taylor series of
// cos and sin there are within 2^-25 with the terms up to x^8 and x^9.  `unit`: kUnit, or NaN.
constexpr float kUnit = 3.6572952e-10f;  // 2 pi 2^-34
__device__ __forceinline__ float2 cos_sin(unsigned long long phase, float sign, float unit) {
  const uint32_t quadrant = (uint32_t)((phase + (1ull << 61)) >> 62);
  const long long rest = (long long)(phase - ((unsigned long long)quadrant << 62));  // within 2^61
  const float x = (float)(int)(rest >> 30) * unit;
  const float z = x * x;
  float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 40320.f, -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
  if (quadrant & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (quadrant & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(c, s * sign);
}

// a^-1/2: of fp32 rows correct to an ulp, of bf16 rows to 2^-22
template <typename T>
__device__ __forceinline__ float inv_sqrt(float a) {
  float y;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(a));
  if constexpr (sizeof(T) == 4) return a < 1e38f && a > 1e-37f ? fmaf(0.5f * y, fmaf(-a * y, y, 1.f), y) : y;
  return y;
}

// Request of token t: start[r] <= t < start[r + 1], r in [0, R) whatever they hold
__device__ __forceinline__ int request_of(const int32_t *start, int R, int t) {
  int lo = 0, hi = R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// of rows with so many columns a lane
constexpr int blocks_per_sm(int cols, int mode) { return (mode == kBwd ? 2 : 4) / (cols > 8 ? 2 : 1); }

// A thread's rows come through shared memory, its own 16-byte pieces in kStages
// slots that only it writes (asynchronously) and reads, so nothing waits but the
// thread itself.  An SM has 128 KB of slots forwards and 64 KB backwards, where two rows
// are read for one that is written: B = 1, H = 64, S = 65,536, D = 128 in bf16 backwards
// 519 us with 48 KB, 559 with 128 KB and 556 with three blocks of 32 KB, where this was
// 490 (485 since: the sum of dw behind it).
template <int CH, int MODE, int COLS>
struct Ring {
  static constexpr int kPieces = CH * (MODE == kBwd ? 2 : 1);  // of a row
  static constexpr int kStages = (MODE == kBwd ? 64 : 128) * 1024 / blocks_per_sm(CH * COLS, MODE) / (kPieces * kThreads * 16);
  static constexpr int kBytes = kStages * kPieces * kThreads * 16;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *p, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A sum in fp32 with what its additions round off beside it (this GPU is slow at doubles).
struct Sum {
  float s, rest;
  __device__ __forceinline__ void add(float x) {
    const float t = s + x, z = t - s;
    rest += (s - (t - z)) + (x - z);
    s = t;
  }
  __device__ __forceinline__ float value() const { return rest == rest ? s + rest : s; }  // rest: NaN of infinite sums
};

// CH chunks of a row a lane, chunks l, l + L, ... for lane l of the row's L: the lanes
// of an access are neighbours in memory (with 8 columns of fp32 side by side a lane
// each 32-byte sector went over the way to L2 in two halves: backward of 2 x 8 x 4,093
// rows of 64 columns 25 us, 19 this way).
template <typename T, int L, int CH, int MODE, bool HALVES>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(CH * 16 / (int)sizeof(T), MODE)) hca_norm_rope_kernel(const Args a) {
  using V = Vec<T, HALVES>;
  using R = Ring<CH, MODE, V::kCols>;
  constexpr int kCols = V::kCols, kSlots = V::kSlots, kF4 = kCols / 4, kCs = HALVES ? kCols : kCols / 2;
  constexpr int kRows = kThreads / L, kRowsLog = L == 8 ? 5 : L == 16 ? 4 : 3;  // rows of a pass
  static_assert(kRows == 1 << kRowsLog, "a power of two");
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, l = tid % L, group = tid / L;
  const int np = a.rot / 2, row_lanes = lane & ~(L - 1);
  const uint32_t ring = tc::smem_u32(smem) + 16 * tid;
  float4 *sh_dw = reinterpret_cast<float4 *>(smem + R::kBytes);                 // [2][CH * kF4][kThreads] (backward)
  unsigned long long *sh_freq =
      reinterpret_cast<unsigned long long *>(smem + R::kBytes + (MODE == kBwd ? 2 * CH * kF4 * kThreads * 16 : 0));  // [axes][np]
  float2 *sh_cs = reinterpret_cast<float2 *>(sh_freq + a.axes * np);            // [tile][np]
  float *sh_w = reinterpret_cast<float *>(sh_cs + a.tile * np);                 // [2][D] weights
  long long *sh_pos = reinterpret_cast<long long *>(sh_w + (MODE == kRope ? 0 : 2 * a.D));  // [axes][tile] coordinates
  int *sh_req = reinterpret_cast<int *>(sh_pos + a.axes * a.tile);              // [2][R + 1] starts and held
  const int token = group & (a.tile - 1), head0 = group >> a.log_tile, head_step = kRows >> a.log_tile, step_log = kRowsLog - a.log_tile;

  if constexpr (MODE == kBwd) tc::pdl_launch_dependents();  // the sums of dw wait for this kernel's end by themselves
  // What all items need, in registers first: the loads' latency passes while the
  // first rows' copies are issued.
  const bool listed = a.start && a.R <= kRequestsInSmem;
  const float freq = tid < a.axes * np ? a.freq[tid] : 0.f;
  float weight[2] = {1.f, 1.f};
  if constexpr (MODE != kRope) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (a.t[i].w && tid < a.D) weight[i] = a.t[i].w[tid];
  }
  int request[2] = {0, 0}, live = a.S;
  if (a.start) {
    if (listed && tid <= a.R) request[0] = a.start[tid];
    if (listed && tid < a.R && a.held) request[1] = a.held[tid];
    live = a.start[a.R];  // rows behind the last request's are left
  }
  int odd = 0;  // one of the thread's frequencies has no angle
  auto keep = [&] {
    odd = no_angle(freq);
    if (tid < a.axes * np) sh_freq[tid] = turns(freq);
    for (int i = tid + kThreads; i < a.axes * np; i += kThreads) {
      const float f = a.freq[i];
      sh_freq[i] = turns(f);
      odd |= no_angle(f);
    }
    if constexpr (MODE != kRope) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (tid < a.D) sh_w[i * a.D + tid] = weight[i];
        for (int d = tid + kThreads; d < a.D; d += kThreads) sh_w[i * a.D + d] = a.t[i].w ? a.t[i].w[d] : 1.f;
      }
    }
    if (listed) {
      if (tid <= a.R) {
        sh_req[tid] = request[0];
        sh_req[a.R + 1 + tid] = request[1];
      }
      for (int i = tid + kThreads; i <= a.R; i += kThreads) {
        sh_req[i] = a.start[i];
        sh_req[a.R + 1 + i] = a.held && i < a.R ? a.held[i] : 0;
      }
    }
    live = min(a.S, live);
  };

  // columns of the lane
  bool mine[CH], turned[CH], upper[CH];
  int partner[CH], pair0[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = l + k * L, z = kCols * c - a.first;  // chunk, its first column among the rotated ones
    mine[k] = kCols * c < a.D;
    turned[k] = mine[k] && z >= 0 && z < a.rot;
    upper[k] = HALVES && z >= np;
    pair0[k] = HALVES ? (upper[k] ? z - np : z) : z / 2;
    partner[k] = turned[k] && HALVES ? (upper[k] ? c - np / kCols : c + np / kCols) : c;
  }
  if constexpr (MODE == kBwd) {
#pragma unroll
    for (int i = 0; i < 2 * CH * kF4; ++i) sh_dw[i * kThreads + tid] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float inv_d = 1.f / (float)a.D;

  const uint32_t items = a.tiles * a.splits;  // below 2^31
  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    const uint32_t tile = item / (uint32_t)a.splits, row = tile / a.per_row;
    const int split = (int)(item - tile * a.splits), b = (int)row, s0 = (int)(tile - row * a.per_row) << a.log_tile;
    const int s = s0 + token;
    const bool there = s < a.S;  // rows behind the last request's are read like others
    long long coordinate = 0;
    if (tid < a.axes * a.tile) {
      const int x = tid >> a.log_tile, at = s0 + (tid & (a.tile - 1));
      if (at < a.S) coordinate = a.pos ? a.pos[((size_t)x * a.B + b) * a.S + at] : at;
    }
    // heads of the block's range: of queries, then of kv
    const int lo0 = split * a.per, hi0 = min(lo0 + a.per, a.t[0].H);
    const int lo1 = max(lo0 - a.t[0].H, 0), hi1 = min(lo0 + a.per - a.t[0].H, a.t[1].H);
    const uint32_t n0 = max((hi0 - lo0 + head_step - 1) >> step_log, 0);
    const uint32_t steps = n0 + (MODE == kRope ? 0 : max((hi1 - lo1 + head_step - 1) >> step_log, 0));
    // rows that the thread has of each: heads lo + head0, + head_step, ...
    const uint32_t own0 = there ? max((hi0 - lo0 - head0 + head_step - 1) >> step_log, 0) : 0;
    const uint32_t own1 = there && MODE != kRope ? max((hi1 - lo1 - head0 + head_step - 1) >> step_log, 0) : 0;

    // The thread's rows in order, their pieces on their way to slot n % kStages.
    const T *next_x = static_cast<const T *>(a.t[0].x), *next_g = static_cast<const T *>(a.t[0].g);
    if (own0 > 0) {
      next_x += b * a.t[0].xb + s * a.t[0].xs + (lo0 + head0) * a.t[0].xh + kCols * l;
      if constexpr (MODE == kBwd) next_g += b * a.t[0].gb + s * a.t[0].gs + (lo0 + head0) * a.t[0].gh + kCols * l;
    }
    int64_t step_x = head_step * a.t[0].xh, step_g = MODE == kBwd ? head_step * a.t[0].gh : 0;
    uint32_t at = 0, left = own0;  // of the next row; rows of this tensor that are left
    auto issue = [&] {
      if (MODE != kRope && at == n0) {  // on to kv
        left = own1;
        next_x = static_cast<const T *>(a.t[1].x);
        next_g = static_cast<const T *>(a.t[1].g);
        if (own1 > 0) {
          next_x += b * a.t[1].xb + s * a.t[1].xs + (lo1 + head0) * a.t[1].xh + kCols * l;
          if constexpr (MODE == kBwd) next_g += b * a.t[1].gb + s * a.t[1].gs + (lo1 + head0) * a.t[1].gh + kCols * l;
        }
        step_x = head_step * a.t[1].xh;
        if constexpr (MODE == kBwd) step_g = head_step * a.t[1].gh;
      }
      if (at < steps) {
        const uint32_t to = ring + (at % R::kStages) * (R::kPieces * kThreads * 16);
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const bool row = left > 0 && mine[k];
          const int col = k == 0 || row ? kCols * k * L : 0;
          cp_async_16(to + k * (kThreads * 16), next_x + col, row ? 16 : 0);
          if constexpr (MODE == kBwd) cp_async_16(to + (CH + k) * (kThreads * 16), next_g + col, row ? 16 : 0);
        }
        if (left > 1) {
          next_x += step_x;
          if constexpr (MODE == kBwd) next_g += step_g;
        }
        left -= left > 0;
      }
      ++at;
      cp_async_commit();
    };
#pragma unroll 1
    for (int n = 0; n < min((int)steps, R::kStages); ++n) issue();
#pragma unroll
    for (uint32_t n = 0; n < R::kStages; ++n)
      if (n >= steps) cp_async_commit();  // empty groups

    if (item == blockIdx.x) keep();
    if (s0 >= live) {
      cp_async_wait<0>();
      continue;
    }
    const bool alive = s < live;
    if (tid < a.axes * a.tile) sh_pos[tid] = coordinate;
    const float unit = __syncthreads_or(odd) ? __int_as_float(0x7fc00000) : kUnit;  // and sh_cs is read no more
    if (a.start && !a.pos && a.held) {  // without held nothing turns
      if (tid < a.tile) {
        const int t = s0 + tid, r = request_of(listed ? sh_req : a.start, a.R, t);
        sh_pos[tid] = listed ? (long long)sh_req[a.R + 1 + r] + t - sh_req[r] : (long long)a.held[r] + t - a.start[r];
      }
      __syncthreads();
    }
    for (int i = tid; i < a.tile * np; i += kThreads) {
      const int t = (int)__umulhi(i, a.inv_np), p = i - t * np;
      unsigned long long phase = (unsigned long long)sh_pos[t] * sh_freq[p];
      for (int x = 1; x < a.axes; ++x) phase += (unsigned long long)sh_pos[x * a.tile + t] * sh_freq[x * np + p];
      sh_cs[i] = cos_sin(phase, a.sign, unit);
    }
    __syncthreads();

    uint32_t n = 0;
#pragma unroll
    for (int which = 0; which < (MODE == kRope ? 1 : 2); ++which) {
      const NormRopeTensor &t = a.t[which];
      const uint32_t end = which ? steps : n0;
      if (n >= end) continue;
      T *y = static_cast<T *>(t.y) + b * t.yb + s * t.ys + ((which ? lo1 : lo0) + head0) * t.yh + kCols * l;
      const int64_t step_y = head_step * t.yh;
      uint32_t rows = which ? own1 : own0;  // that are left
      // What a column and its partner count in a rotated column (backwards: turned
      // back).  Forwards the weights are in them.
      uint64_t own[CH][kSlots], other[CH][kSlots], w[CH][kSlots], dw[CH][kSlots];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float2 cs[kCs];
        float wt[kCols], wp[kCols];  // weights of the columns, of their partners
#pragma unroll
        for (int c = 0; c < kCs; ++c) cs[c] = make_float2(1.f, 0.f);
        if (turned[k]) {
#pragma unroll
          for (int c = 0; c < kCs; c += 2) {
            const float4 v = *reinterpret_cast<const float4 *>(sh_cs + token * np + pair0[k] + c);
            cs[c] = make_float2(v.x, v.y);
            cs[c + 1] = make_float2(v.z, v.w);
          }
        }
#pragma unroll
        for (int c = 0; c < kCols; ++c) wt[c] = wp[c] = 1.f;
        if (MODE != kRope && mine[k]) {
          const float *weight = sh_w + which * a.D;
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            *reinterpret_cast<float4 *>(wt + c) = *reinterpret_cast<const float4 *>(weight + kCols * (l + k * L) + c);
            if (HALVES && MODE == kFwd) *reinterpret_cast<float4 *>(wp + c) = *reinterpret_cast<const float4 *>(weight + kCols * partner[k] + c);
          }
        }
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          float o[2], p[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c = V::column(i, e);
            const float2 turn = cs[HALVES ? c : c >> 1];
            const bool second = HALVES ? upper[k] : (c & 1) != 0;
            o[e] = turn.x;
            p[e] = (second == (MODE != kBwd)) ? turn.y : -turn.y;
            if (MODE == kFwd) {
              o[e] *= wt[c];
              p[e] *= HALVES ? wp[c] : wt[c ^ 1];
            }
          }
          own[k][i] = pair(o[0], o[1]);
          other[k][i] = pair(p[0], p[1]);
          w[k][i] = pair(wt[V::column(i, 0)], wt[V::column(i, 1)]);
        }
#pragma unroll
        for (int i = 0; i < kSlots; ++i) dw[k][i] = 0;
      }
      // own f + other f of the partner, for a row's slots
      auto rotate = [&](const V (&v)[CH], const uint64_t (&f)[CH][kSlots], uint64_t (&o)[CH][kSlots]) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          uint64_t q[kSlots];
          if constexpr (HALVES) {
            const int from = row_lanes + (partner[k] & (L - 1));
            V p = v[0].of(from);
#pragma unroll
            for (int j = 1; j < CH; ++j) {  // the partner may be in another chunk of its lane
              const V pj = v[j].of(from);
              if (partner[k] >= j * L) p = pj;
            }
            p.get(q);
          }
#pragma unroll
          for (int i = 0; i < kSlots; ++i) o[k][i] = tc::ffma2(f[k][i], own[k][i], tc::fmul2(HALVES ? q[i] : f[k][i ^ (kSlots / 2)], other[k][i]));
        }
      };
#pragma unroll 1
      for (; n < end; ++n) {
        cp_async_wait<R::kStages - 1>();
        V vx[CH], vg[CH];
        const uint8_t *from = smem + (n % R::kStages) * (R::kPieces * kThreads * 16) + 16 * tid;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          vx[k].load(*reinterpret_cast<const uint4 *>(from + k * (kThreads * 16)));
          if constexpr (MODE == kBwd) vg[k].load(*reinterpret_cast<const uint4 *>(from + (CH + k) * (kThreads * 16)));
        }
        const bool row = alive && rows > 0;
        uint64_t f[CH][kSlots], o[CH][kSlots];
#pragma unroll
        for (int k = 0; k < CH; ++k) vx[k].get(f[k]);
        if constexpr (MODE == kRope) {
          rotate(vx, f, o);
        } else {
          uint64_t ss = 0, hx = 0, gx[CH][kSlots];
          if constexpr (MODE == kBwd) {
            uint64_t g0[CH][kSlots];
#pragma unroll
            for (int k = 0; k < CH; ++k) vg[k].get(g0[k]);
            rotate(vg, g0, o);
          }
#pragma unroll
          for (int k = 0; k < CH; ++k) {
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
              ss = tc::ffma2(f[k][i], f[k][i], ss);
              if constexpr (MODE == kBwd) {
                gx[k][i] = tc::fmul2(o[k][i], f[k][i]);
                hx = tc::ffma2(gx[k][i], w[k][i], hx);
              }
            }
          }
          float s1 = total(ss), h1 = MODE == kBwd ? total(hx) : 0.f;
#pragma unroll
          for (int d = L / 2; d > 0; d >>= 1) {
            s1 += __shfl_xor_sync(0xffffffffu, s1, d);
            if constexpr (MODE == kBwd) h1 += __shfl_xor_sync(0xffffffffu, h1, d);
          }
          const float r = inv_sqrt<T>(fmaf(s1, inv_d, a.eps));
          const uint64_t r2 = pair(r, r);
          if constexpr (MODE == kFwd) {
            rotate(vx, f, o);
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
              for (int i = 0; i < kSlots; ++i) o[k][i] = tc::fmul2(o[k][i], r2);
          } else {
            const float q = -(r * r) * (h1 * inv_d), rw = row ? r : 0.f;
            const uint64_t q2 = pair(q, q), rw2 = pair(rw, rw);
#pragma unroll
            for (int k = 0; k < CH; ++k) {
#pragma unroll
              for (int i = 0; i < kSlots; ++i) {
                dw[k][i] = tc::ffma2(gx[k][i], rw2, dw[k][i]);
                o[k][i] = tc::fmul2(r2, tc::ffma2(f[k][i], q2, tc::fmul2(o[k][i], w[k][i])));
              }
            }
          }
        }
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          if (row && mine[k]) {
            V out;
            out.put(o[k]);
            if (MODE == kRope && !turned[k]) out = vx[k];  // as it was, infinities too
            out.store(y + kCols * k * L);
          }
        }
        y += step_y;
        rows -= rows > 0;
        issue();
      }
      if constexpr (MODE == kBwd) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
#pragma unroll
          for (int i = 0; i < kF4; ++i) {
            float4 &to = sh_dw[((which * CH + k) * kF4 + i) * kThreads + tid], v;
            tc::f32x2_split(dw[k][2 * i], v.x, v.y);
            tc::f32x2_split(dw[k][2 * i + 1], v.z, v.w);
            to = make_float4(to.x + v.x, to.y + v.y, to.z + v.z, to.w + v.w);
          }
        }
      }
    }
    cp_async_wait<0>();  // empty groups, but the next item's are counted anew
  }

  if constexpr (MODE == kBwd) {
    // sums of the block's rows: over its row groups, in their order.  (A thread adds up an
    // item's rows, then the items': one long sum loses a bit for every doubling.)
    __syncthreads();
    for (int i = tid; i < 2 * a.D; i += kThreads) {
      const int which = i / a.D, d = i - which * a.D, chunk = d / kCols, c = d % kCols;
      if (!a.t[which].dw) continue;
      int slot = 0;  // of the column among the chunk's floats
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        if (V::column(j >> 1, j & 1) == c) slot = j;
      const float *from = reinterpret_cast<const float *>(sh_dw + (size_t)((which * CH + chunk / L) * kF4 + (slot >> 2)) * kThreads + chunk % L) + (slot & 3);
      Sum v = {0.f, 0.f};
#pragma unroll 8
      for (int r = 0; r < kRows; ++r) v.add(from[4 * r * L]);
      a.part[((size_t)blockIdx.x * 2 + which) * a.D + d] = v.value();
    }
  }
}

// dw from the blocks' sums, in a fixed order: 32 warps take every 32nd block each,
// a lane a column.  (In doubles 6 us longer: backward of 2 x 8 x 4,093 fp32 rows of 64
// columns 17.7 us, 12.1 this way.)
constexpr int kDwThreads = 1024;
__global__ void __launch_bounds__(kDwThreads) hca_norm_rope_dw_kernel(const float *part, int n, int D, float *dwq, float *dwkv) {
  __shared__ Sum sum[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y, d = blockIdx.x * 32 + lane;
  float *dw = which ? dwkv : dwq;
  tc::pdl_wait();
  if (!dw) return;
  Sum v = {0.f, 0.f};
  if (d < D) {
#pragma unroll 8
    for (int i = warp; i < n; i += 32) v.add(part[((size_t)i * 2 + which) * D + d]);
  }
  sum[warp][lane] = v;
  __syncthreads();
  // the 32 sums of column `warp` by the warp's lanes
  v = sum[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float s = __shfl_xor_sync(0xffffffffu, v.s, o), rest = __shfl_xor_sync(0xffffffffu, v.rest, o);
    v.add(s);
    v.rest += rest;
  }
  if (lane == 0 && blockIdx.x * 32 + warp < D) dw[blockIdx.x * 32 + warp] = v.value();
}

template <typename T, int L, int CH, int MODE, bool HALVES>
cudaError_t launch(Args &a, cudaStream_t st) {
  constexpr int kRows = kThreads / L, kPerSm = blocks_per_sm(CH * 16 / (int)sizeof(T), MODE), kBegin = MODE == kRope ? 3 : 8;
  const int sms = tc::sm_count();
  if (sms <= 0) return cudaErrorNoDevice;
  // a tile's tokens: those of a pass, or as few as there are
  a.tile = 1, a.log_tile = 0;
  while (a.tile < kRows && a.tile < a.S) a.tile *= 2, ++a.log_tile;
  a.per_row = (a.S + a.tile - 1) >> a.log_tile;
  a.tiles = a.B * a.per_row;
  a.inv_np = a.rot > 0 ? 0xffffffffu / (uint32_t)(a.rot / 2) + 1 : 0;
  // Head ranges: all heads of a tile in one block, or more blocks where there would be
  // too few.  A block costs its rows and a beginning of kBegin rows' time; the blocks
  // that the SMs hold at once run together.
  const int heads = a.t[0].H + a.t[1].H, pass = kRows >> a.log_tile, at_once = kPerSm * sms;
  long long least = 0;
  a.per = heads;
  for (int splits = 1; splits <= heads; ++splits) {
    const int per = ((heads + splits - 1) / splits + pass - 1) / pass * pass;
    const long long blocks = (long long)a.tiles * ((heads + per - 1) / per), cost = (blocks + at_once - 1) / at_once * (kBegin + per / pass);
    if (splits == 1 || cost < least) least = cost, a.per = per;
    if (blocks > 8ll * at_once) break;
  }
  a.splits = (heads + a.per - 1) / a.per;
  using R = Ring<CH, MODE, 16 / (int)sizeof(T)>;
  constexpr int kFixed = R::kBytes + (MODE == kBwd ? 2 * CH * (4 / (int)sizeof(T)) * kThreads * 16 : 0);
  size_t smem = kFixed + 8 * ((size_t)(a.axes + a.tile) * (a.rot / 2) + a.axes * a.tile) + (MODE == kRope ? 0 : 8 * (size_t)a.D);
  if (a.start && a.R <= kRequestsInSmem) smem += 2 * sizeof(int) * ((size_t)a.R + 1);
  auto *kernel = hca_norm_rope_kernel<T, L, CH, MODE, HALVES>;
  static tc::SmemAttrOnce attr;
  cudaError_t e = attr.ensure(reinterpret_cast<const void *>(kernel), kFixed + 38 * 1024);  // the most that the rest takes
  if (e != cudaSuccess) return e;
  uint32_t grid = a.tiles * a.splits;
  // Blocks that take item after item: backwards, since each leaves a part of dw, and
  // where two of them fill an SM and have few rows a thread (forward of 540 MB of rows of
  // 512 columns: one head 153 us, 197 with a block an item; 8 heads 88 and 92; 16 heads
  // 97 and 85.  With four an SM and 128 columns one head 218 and 229, 8 heads 95 and 94).
  const bool stay = MODE == kBwd || (kPerSm <= 2 && a.per <= 12 * pass);
  if (stay) grid = std::min<uint32_t>(grid, std::min(kNormRopeParts, kPerSm * sms));
  ProfScope prof(MODE == kBwd ? kKNormRopeBwd : kKNormRope, st);
  kernel<<<grid, kThreads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (MODE == kBwd && (a.t[0].dw || a.t[1].dw)) {
    e = cache::launch_behind(hca_norm_rope_dw_kernel, dim3((a.D + 31) / 32, 2), kDwThreads, 0, st, (const float *)a.part, (int)grid, a.D, a.t[0].dw,
                             a.t[1].dw);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int MODE, bool HALVES>
cudaError_t by_width(Args &a, cudaStream_t st) {
  constexpr int kCh = (int)sizeof(T) / 2;  // chunks of 8 columns
  if (a.D <= 64) return launch<T, 8, kCh, MODE, HALVES>(a, st);
  if (a.D <= 128) return launch<T, 16, kCh, MODE, HALVES>(a, st);
  if (a.D <= 256) return launch<T, 32, kCh, MODE, HALVES>(a, st);
  return launch<T, 32, 2 * kCh, MODE, HALVES>(a, st);
}

template <int MODE>
cudaError_t by_type(Args &a, int dtype, bool halves, cudaStream_t st) {
  if (dtype == HCA_F32) return halves ? by_width<float, MODE, true>(a, st) : by_width<float, MODE, false>(a, st);
  return halves ? by_width<__nv_bfloat16, MODE, true>(a, st) : by_width<__nv_bfloat16, MODE, false>(a, st);
}

}  // namespace

cudaError_t norm_rope(const NormRopeArgs &n, cudaStream_t st) {
  Args a;
  a.t[0] = n.t[0];
  a.t[1] = n.t[1];
  a.pos = n.pos; a.start = n.start; a.held = n.held; a.freq = n.freq; a.part = n.part;
  a.B = n.B; a.S = n.S; a.D = n.D; a.R = n.R; a.axes = n.axes; a.first = n.first; a.rot = n.rot;
  a.sign = n.inverse ? -1.f : 1.f;
  a.eps = n.eps;
  switch (n.mode) {
    case 0: return by_type<kRope>(a, n.dtype, n.halves, st);
    case 1: return by_type<kFwd>(a, n.dtype, n.halves, st);
    default: return by_type<kBwd>(a, n.dtype, n.halves, st);
  }
}

}  // namespace hca
