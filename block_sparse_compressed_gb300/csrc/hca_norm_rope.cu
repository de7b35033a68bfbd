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
// per unit, F = f / 2pi * 2^64 mod 2^64 (in two doubles, exact to 2^-64 turns),
// and a phase is sum_a c_a F[a] in integers, where the wrap-around of 64 bits is
// the reduction to one turn: off by 2^-33 turns at most for any 32-bit
// coordinates.  The two upper bits (rounded) are the quadrant, the rest, an eighth
// of a turn at most, goes through sincospif.
//
// A row belongs to L neighbouring lanes, 8 consecutive columns (one or two 16-byte
// accesses) a lane and chunk, so a row is read once, stays in registers between
// the sum of its squares and its output, and is written once.  A block takes a
// tile of tokens and a range of heads: the tile's cos and sin are made once in
// shared memory, then each lane keeps those of its own columns and token in
// registers for all of the block's heads.
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
  long long tiles;      // token tiles of all batch rows
  int tile, log_tile;   // tokens of a tile, a power of two
  int splits, per;      // head ranges of a tile, heads (of q, then kv) of a range
};

template <typename T>
struct Vec {  // 8 columns
  static constexpr int kWords = sizeof(T) * 2;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T *p) {
    const uint4 *v = reinterpret_cast<const uint4 *>(p);
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 u = v[i];
      w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
};

__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(tc::pack_bf16x2(f[0], f[1]), tc::pack_bf16x2(f[2], f[3]),
                                             tc::pack_bf16x2(f[4], f[5]), tc::pack_bf16x2(f[6], f[7]));
}

// f / 2pi of a turn per unit as a 64-bit fraction
__device__ __forceinline__ unsigned long long turns(float f) {
  // 1 / 2pi in two doubles
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  const double p = (double)f * kHi;
  const double e = fma((double)f, kHi, -p) + (double)f * kLo;
  const double q = p - rint(p);  // exact
  // the sum is taken mod 2^64, so half a turn is the same upwards and downwards
  return (unsigned long long)__double2ll_rn(q * 18446744073709551616.0) + (unsigned long long)__double2ll_rn(e * 18446744073709551616.0);
}

__device__ __forceinline__ float2 cos_sin(unsigned long long phase, float sign) {
  const uint32_t quadrant = (uint32_t)((phase + (1ull << 61)) >> 62);
  const long long rest = (long long)(phase - ((unsigned long long)quadrant << 62));  // within 2^61
  float s, c;
  sincospif((float)(int)(rest >> 30) * 1.1641532182693481e-10f /* 2^-33 */, &s, &c);
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

// a^-1/2, correct to an ulp
__device__ __forceinline__ float inv_sqrt(float a) {
  const float y = rsqrtf(a);
  return a < 1e38f && a > 1e-37f ? fmaf(0.5f * y, fmaf(-a * y, y, 1.f), y) : y;
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

template <int CH>
struct Turn {
  float c[CH][8], s[CH][8];  // halves: of each column; interleaved: of pair k in [k], k < 4
};

template <typename T, int L, int CH, int MODE, bool HALVES>
__global__ void __launch_bounds__(kThreads) hca_norm_rope_kernel(const Args a) {
  constexpr int kRows = kThreads / L;  // rows of a pass
  constexpr int kBatch = CH > 1 || MODE == kBwd ? 2 : 4;  // rows of a lane in flight
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, l = tid % L, group = tid / L;
  const int np = a.rot / 2, row_lanes = lane & ~(L - 1);
  unsigned long long *sh_freq = reinterpret_cast<unsigned long long *>(smem);   // [axes][np]
  float2 *sh_cs = reinterpret_cast<float2 *>(sh_freq + a.axes * np);            // [tile][np]
  long long *sh_pos = reinterpret_cast<long long *>(sh_cs + a.tile * np);       // [tile] positions from start and held
  int *sh_req = reinterpret_cast<int *>(sh_pos + a.tile);                       // [2][R + 1] starts and held
  const int token = group & (a.tile - 1), head0 = group >> a.log_tile, head_step = kRows >> a.log_tile;

  for (int i = tid; i < a.axes * np; i += kThreads) sh_freq[i] = turns(a.freq[i]);
  int live = a.S;
  const bool listed = a.start && a.R <= kRequestsInSmem;
  if (a.start) {
    if (listed) {
      for (int i = tid; i <= a.R; i += kThreads) {
        sh_req[i] = a.start[i];
        sh_req[a.R + 1 + i] = a.held && i < a.R ? a.held[i] : 0;
      }
    }
    live = min(a.S, a.start[a.R]);  // rows behind the last request's are left
  }

  // columns of the lane
  bool mine[CH], turned[CH];
  int partner[CH], pair0[CH];
  bool upper[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = l + k * L, z = 8 * c - a.first;  // chunk, its first column among the rotated ones
    mine[k] = 8 * c < a.D;
    turned[k] = mine[k] && z >= 0 && z < a.rot;
    upper[k] = HALVES && z >= np;
    pair0[k] = HALVES ? (upper[k] ? z - np : z) : z / 2;
    partner[k] = turned[k] && HALVES ? (upper[k] ? c - np / 8 : c + np / 8) : c;
  }
  float dw[2][CH][8];
  if constexpr (MODE == kBwd) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][k][j] = 0.f;
  }
  const float inv_d = 1.f / (float)a.D;

  for (long long item = blockIdx.x; item < a.tiles * a.splits; item += gridDim.x) {
    const int split = (int)(item % a.splits);
    const long long tile = item / a.splits;
    const int per_row = (a.S + a.tile - 1) >> a.log_tile;
    const int b = (int)(tile / per_row), s0 = (int)(tile % per_row) << a.log_tile;
    if (s0 >= live) continue;
    __syncthreads();  // sh_cs may still be read; sh_freq and sh_req are written
    if (a.start && !a.pos) {
      if (tid < a.tile) {
        const int s = s0 + tid, r = request_of(listed ? sh_req : a.start, a.R, s);
        sh_pos[tid] = listed ? (long long)sh_req[a.R + 1 + r] + s - sh_req[r] : (long long)a.held[r] + s - a.start[r];
      }
      __syncthreads();
    }
    for (int i = tid; i < a.tile * np; i += kThreads) {
      const int t = i / np, p = i - t * np, s = s0 + t;
      unsigned long long phase = 0;
      if (s < live) {
        if (a.pos) {
          for (int x = 0; x < a.axes; ++x)
            phase += (unsigned long long)(long long)a.pos[((size_t)x * a.B + b) * a.S + s] * sh_freq[x * np + p];
        } else {
          phase = (unsigned long long)(a.start ? sh_pos[t] : s) * sh_freq[p];
        }
      }
      sh_cs[i] = cos_sin(phase, a.sign);
    }
    __syncthreads();
    Turn<CH> turn;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
#pragma unroll
      for (int j = 0; j < (HALVES ? 8 : 4); ++j) {
        const float2 v = turned[k] ? sh_cs[token * np + pair0[k] + j] : make_float2(1.f, 0.f);
        turn.c[k][j] = v.x;
        turn.s[k][j] = HALVES && !upper[k] ? -v.y : v.y;
      }
    }
    const int s = s0 + token;
    const bool alive = s < live;

    // in place: (u, v) of each pair turned by the angle (by minus it for back)
    auto rotate = [&](float (&f)[CH][8], auto back) {
      constexpr float kSign = decltype(back)::value ? -1.f : 1.f;
      if constexpr (HALVES) {
        float o[CH][8];
#pragma unroll
        for (int k = 0; k < CH; ++k) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float p;
            if constexpr (CH == 1) {
              p = __shfl_sync(0xffffffffu, f[0][j], row_lanes + partner[0]);
            } else {
              // the partner may be in the other chunk of its lane
              const float p0 = __shfl_sync(0xffffffffu, f[0][j], partner[k] & 31), p1 = __shfl_sync(0xffffffffu, f[1][j], partner[k] & 31);
              p = partner[k] >= 32 ? p1 : p0;
            }
            o[k][j] = turned[k] ? fmaf(f[k][j], turn.c[k][j], kSign * p * turn.s[k][j]) : f[k][j];
          }
        }
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) f[k][j] = o[k][j];
      } else {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float u = f[k][2 * j], v = f[k][2 * j + 1], c = turn.c[k][j], sn = kSign * turn.s[k][j];
            if (turned[k]) {
              f[k][2 * j] = fmaf(u, c, -v * sn);
              f[k][2 * j + 1] = fmaf(v, c, u * sn);
            }
          }
        }
      }
    };

#pragma unroll
    for (int which = 0; which < (MODE == kRope ? 1 : 2); ++which) {
      const NormRopeTensor &t = a.t[which];
      // heads of the block's range
      const int base = which ? a.t[0].H : 0;
      const int h_lo = max(split * a.per - base, 0), h_hi = min(min((split + 1) * a.per, base + t.H) - base, t.H);
      if (h_lo >= h_hi) continue;
      const T *x = static_cast<const T *>(t.x) + b * t.xb + s * t.xs + 8 * l;
      const T *g = MODE == kBwd ? static_cast<const T *>(t.g) + b * t.gb + s * t.gs + 8 * l : nullptr;
      T *y = static_cast<T *>(t.y) + b * t.yb + s * t.ys + 8 * l;
      float w[CH][8];
      if constexpr (MODE != kRope) {
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) w[k][j] = t.w && mine[k] ? t.w[8 * (l + k * L) + j] : 1.f;
      }
#pragma unroll 1
      for (int h0 = h_lo; h0 < h_hi; h0 += kBatch * head_step) {
        Vec<T> vx[kBatch][CH], vg[kBatch][CH];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int h = h0 + u * head_step + head0;
#pragma unroll
          for (int k = 0; k < CH; ++k) {
            if (alive && h < h_hi && mine[k]) {
              vx[u][k].load(x + h * t.xh + 8 * k * L);
              if constexpr (MODE == kBwd) vg[u][k].load(g + h * t.gh + 8 * k * L);
            } else {
              vx[u][k].zero();
              if constexpr (MODE == kBwd) vg[u][k].zero();
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int h = h0 + u * head_step + head0;
          float f[CH][8];
#pragma unroll
          for (int k = 0; k < CH; ++k) vx[u][k].get(f[k]);
          if constexpr (MODE == kRope) {
            rotate(f, std::false_type());
          } else {
            float ss = 0.f, hx = 0.f;
            float gr[CH][8];
            if constexpr (MODE == kBwd) {
#pragma unroll
              for (int k = 0; k < CH; ++k) vg[u][k].get(gr[k]);
              rotate(gr, std::true_type());
            }
#pragma unroll
            for (int k = 0; k < CH; ++k) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                ss = fmaf(f[k][j], f[k][j], ss);
                if constexpr (MODE == kBwd) hx = fmaf(gr[k][j] * w[k][j], f[k][j], hx);
              }
            }
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) {
              ss += __shfl_xor_sync(0xffffffffu, ss, o);
              if constexpr (MODE == kBwd) hx += __shfl_xor_sync(0xffffffffu, hx, o);
            }
            const float r = inv_sqrt(fmaf(ss, inv_d, a.eps));
            if constexpr (MODE == kFwd) {
#pragma unroll
              for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) f[k][j] = f[k][j] * r * w[k][j];
              rotate(f, std::false_type());
            } else {
              const float q = r * r * (hx * inv_d);
              const bool row = alive && h < h_hi;
#pragma unroll
              for (int k = 0; k < CH; ++k) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const float xv = f[k][j], gv = gr[k][j];
                  if (row) dw[which][k][j] = fmaf(gv * xv, r, dw[which][k][j]);
                  f[k][j] = r * fmaf(-xv, q, gv * w[k][j]);
                }
              }
            }
          }
#pragma unroll
          for (int k = 0; k < CH; ++k)
            if (alive && h < h_hi && mine[k]) store8(y + h * t.yh + 8 * k * L, f[k]);
        }
      }
    }
  }

  if constexpr (MODE == kBwd) {
    // sums of the block's rows: over its row groups in shared memory, in their order
    float *sum = reinterpret_cast<float *>(smem);  // [kRows][D]
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if (!a.t[which].dw) continue;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < CH; ++k)
        if (mine[k]) store8(sum + (size_t)group * a.D + 8 * (l + k * L), dw[which][k]);
      __syncthreads();
      for (int d = tid; d < a.D; d += kThreads) {
        float v = 0.f;
#pragma unroll 8
        for (int i = 0; i < kRows; ++i) v += sum[(size_t)i * a.D + d];
        a.part[((size_t)blockIdx.x * 2 + which) * a.D + d] = v;
      }
    }
  }
}

// dw from the blocks' sums, in a fixed order: 8 warps take every 8th block each,
// a lane a column.
__global__ void __launch_bounds__(kThreads) hca_norm_rope_dw_kernel(const float *part, int n, int D, float *dwq, float *dwkv) {
  __shared__ float sum[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y, d = blockIdx.x * 32 + lane;
  float *dw = which ? dwkv : dwq;
  tc::pdl_wait();
  if (!dw) return;
  float v = 0.f;
  if (d < D) {
#pragma unroll 8
    for (int i = warp; i < n; i += 8) v += part[((size_t)i * 2 + which) * D + d];
  }
  sum[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && d < D) {
    for (int i = 1; i < 8; ++i) v += sum[i][lane];
    dw[d] = v;
  }
}

template <typename T, int L, int CH, int MODE, bool HALVES>
cudaError_t launch(Args &a, cudaStream_t st) {
  constexpr int kRows = kThreads / L;
  const int sms = tc::sm_count();
  if (sms <= 0) return cudaErrorNoDevice;
  // a tile's tokens: those of a pass, or as few as there are
  a.tile = 1, a.log_tile = 0;
  while (a.tile < kRows && a.tile < a.S) a.tile *= 2, ++a.log_tile;
  a.tiles = (long long)a.B * ((a.S + a.tile - 1) >> a.log_tile);
  const int heads = a.t[0].H + a.t[1].H, pass = kRows >> a.log_tile;
  const int want = (int)std::min<long long>((4ll * sms + a.tiles - 1) / a.tiles, heads);
  a.per = ((heads + want - 1) / want + pass - 1) / pass * pass;
  a.splits = (heads + a.per - 1) / a.per;
  size_t smem = 8 * ((size_t)(a.axes + a.tile) * (a.rot / 2) + a.tile);  // 33 KB at most, with the requests
  if (a.start && a.R <= kRequestsInSmem) smem += 2 * sizeof(int) * ((size_t)a.R + 1);
  if (MODE == kBwd) smem = std::max(smem, (size_t)kRows * a.D * sizeof(float));
  long long grid = a.tiles * a.splits;
  grid = std::min<long long>(grid, MODE == kBwd ? std::min(kNormRopeParts, 4 * sms) : 1 << 30);
  ProfScope prof(MODE == kBwd ? kKNormRopeBwd : kKNormRope, st);
  hca_norm_rope_kernel<T, L, CH, MODE, HALVES><<<(unsigned)grid, kThreads, smem, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (MODE == kBwd && (a.t[0].dw || a.t[1].dw)) {
    e = cache::launch_behind(hca_norm_rope_dw_kernel, dim3((a.D + 31) / 32, 2), kThreads, 0, st, (const float *)a.part, (int)grid, a.D, a.t[0].dw,
                             a.t[1].dw);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int MODE, bool HALVES>
cudaError_t by_width(Args &a, cudaStream_t st) {
  if (a.D <= 64) return launch<T, 8, 1, MODE, HALVES>(a, st);
  if (a.D <= 128) return launch<T, 16, 1, MODE, HALVES>(a, st);
  if (a.D <= 256) return launch<T, 32, 1, MODE, HALVES>(a, st);
  return launch<T, 32, 2, MODE, HALVES>(a, st);
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
