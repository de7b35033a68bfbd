// hca_cache_attn_tc.cu -- attention over the 8-bit cache on the tensor cores
// (tcgen05 + TMEM + TMA), bf16 queries, D = 64 or 128.
//
// A CTA takes a range of the line of tiles (hca_cache.cuh).  A tile is 128 keys
// of one group, a group NQ columns: up to P positions x HS heads of a request.
// With the keys in the M dimension nothing is wasted when a request brings one
// token and few heads:
//   S^T [keys x NQ]   = K  [128 x D]    (Q_hi | Q_lo)^T       kind::f8f6f4
//   O^T [D x 2 NQ]   += K^T [D x 128]   (P_hi | P_lo)         kind::f8f6f4
// The cache's e4m3 rows go from TMA to the tensor cores as they are, once as
// K-major and once as MN-major operand; nothing is converted on the way, and
// each key's block scale multiplies its scores and its probabilities.
//
// Eight bits on the other side would be too few, so q and the probabilities are
// each the sum of two e4m3 numbers.  An e4m3 number has 4 significant bits and
// the rest after rounding to it has 4 more: a bf16 q (8 bits) is exact as q_hi +
// q_lo of one power-of-two scale for the whole tile, but for values below 2^-17
// of the tile's largest (both products go to the same accumulator).  P_hi + P_lo
// / 32 is P to 8 bits; the two have accumulators of their own, joined in the
// epilogue, so that P_lo can be 2^5 larger and small probabilities keep their
// bits down to 2^-20 of the largest.  At twice the rate of bf16 the two products
// cost what one bf16 product would, and no operand is converted or staged again.
//
// Softmax.  Thread k of the softmax warps owns key k: it reads S^T's row k
// (NQ scores in its lane), so a column's maximum lies across threads.  Instead
// of reducing every column of every tile, a column keeps a reference: the
// maximum of the first tile that it sees, placed at 2^5.  A tile whose scores
// stay below 2^8 uses it as it is (one vote for the tile); else the column
// maxima are taken, references move and O is rescaled.  Row sums are kept per
// thread in fp32 and joined once, at the end of the group.
//
// A row that some column does not see may hold anything, and 0 * NaN is not 0:
// its thread zeroes it in shared memory between the two products if no column
// sees it, or if it holds a NaN (whoever sees it has a NaN for a probability).
#include <cuda_bf16.h>

#include "hca_cache_attn.cuh"
#include "tc_tiles.cuh"

namespace hca {
using namespace tc;
using namespace cache;

namespace {

constexpr float kRefLog2 = 5.f;   // a reference maximum's probability is 2^5
constexpr float kTopLog2 = 8.f;   // larger ones move the reference (e4m3 ends at 448)

template <int NQ, int D>
struct Cfg {
  static constexpr int WG = NQ == 128 ? 2 : 1;         // softmax warpgroups, CW columns each
  static constexpr int CW = NQ / WG;
  static constexpr int kSoft = 128 * WG;               // softmax threads
  static constexpr int kThreads = kSoft + 64;          // and a TMA and an MMA warp
  static constexpr int kCtas = NQ == 128 ? 1 : 2;      // CTAs per SM
  static constexpr int kStageBytes = kTileKeys * D;
  static constexpr int kStages = (NQ == 128 ? 6 : 3) * (128 / D);
  static constexpr int kQBytes = 2 * NQ * D;           // q_hi | q_lo
  static constexpr int kPHalf = NQ == 128 ? 16384 : 0; // P_lo's own 128-byte rows for 128 columns
  static constexpr int kPBytes = 16384 + kPHalf;       // one of two P buffers
  static constexpr int kOffQ = kStages * kStageBytes;
  static constexpr int kOffP = kOffQ + (kQBytes < 1024 ? 1024 : kQBytes);
  static constexpr int kSmem = kOffP + 2 * kPBytes + 1024;
  static constexpr int kTmem = 4 * NQ;                 // S twice, O_hi, O_lo
};

struct __align__(16) PageMeta {
  int key0;     // first key of the page
  int kind;     // 0 raw, 1 compressed, 2 no page
  float scale, log2_scale;
};

template <int NQ, int D>
struct Shared {
  using C = Cfg<NQ, D>;
  uint64_t kv_full[C::kStages], kv_empty[C::kStages];
  uint64_t q_full, s_full[2], s_free[2], p_full[2], pv_done[2], drain, never;
  PageMeta meta[C::kStages][8];
  int wmax[4 * C::WG][C::CW];
  float lred[4 * C::WG][C::CW];
  __align__(16) float nref[NQ];  // read four at a time
  float delta[NQ], fac[NQ], inv[NQ];
  int unset[NQ];
  float amax[4 * C::WG];
  uint32_t tmem_base;
  int abort, first;
};

// Order-preserving map of floats to ints (NaN above +inf).
__device__ __forceinline__ int ordered(float f) {
  const int i = __float_as_int(f);
  return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff); }

// N values per lane -> lane l's own column l (mod N) summed over the warp.
template <int N>
__device__ __forceinline__ float column_sum(float (&v)[N], int lane) {
#pragma unroll
  for (int o = N / 2; o >= 1; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  float s = v[0];
#pragma unroll
  for (int o = N; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// CW consecutive TMEM columns of this thread's lane.
template <int N>
__device__ __forceinline__ void load_cols(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 16) {
    tmem_ld16(addr, r);
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 32) tmem_ld32(addr + c, *reinterpret_cast<uint32_t(*)[32]>(&r[c]));
  }
  tmem_wait_ld();
}

__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two values to two e4m3 numbers each: hi = e4m3(v), lo = e4m3((v - hi) * f).
// fp16 holds v to 11 bits, hi and the difference exactly.
__device__ __forceinline__ void split2(uint32_t h2, uint32_t f2, uint32_t &hi, uint32_t &lo) {
  hi = e4m3x2_from_f16x2(h2);
  lo = e4m3x2_from_f16x2(hmul2(hsub2(h2, f16x2_from_e4m3x2(hi)), f2));
}

template <int NQ, int D>
__global__ void __launch_bounds__(Cfg<NQ, D>::kThreads, Cfg<NQ, D>::kCtas)
    hca_cache_attn_kernel(const __grid_constant__ CUtensorMap map_raw, const __grid_constant__ CUtensorMap map_comp,
                          const AttnParams p) {
  using C = Cfg<NQ, D>;
  constexpr int CW = C::CW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Shared<NQ, D> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int *abort_flag = &sh.abort;
  int32_t *status = &p.hdr->status;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh.kv_full[s], 2);  // the expected bytes, then the pages' data
      mbar_init(&sh.kv_empty[s], 1);
    }
    mbar_init(&sh.q_full, C::kSoft);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.s_full[b], 1);
      mbar_init(&sh.s_free[b], C::kSoft);
      mbar_init(&sh.p_full[b], C::kSoft);
      mbar_init(&sh.pv_done[b], 1);
    }
    mbar_init(&sh.drain, 1);
    mbar_init(&sh.never, 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  const long long ntiles = p.hdr->ntiles;
  const long long quota = cta_quota(ntiles, p.grid, kMinTiles);
  const long long c0 = quota * blockIdx.x, c1 = min(c0 + quota, ntiles);
  const bool busy = c0 < c1;
  if (warp == 0) {
    tmem_alloc(&sh.tmem_base, C::kTmem);
    tmem_relinquish();
  }
  if (warp == C::kSoft / 32 && busy) {
    const int g = find_group(p.groups, p.hdr->ngroups, c0);
    if (lane == 0) sh.first = p.first[blockIdx.x] = g;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  if (warp == C::kSoft / 32) {
    // -------------------------------------------------------------- TMA
    if (busy) {
      if (lane == 0) {
        tma_prefetch_map(&map_raw);
        tma_prefetch_map(&map_comp);
      }
      const int ppt = kTileKeys >> p.log_bs;  // pages per tile: a power of two, 1 .. 8
      const int batch = 32 / ppt;             // tiles whose pages the warp's lanes look up at once
      const int page_bytes = D << p.log_bs;
      uint32_t n = 0, issued = 0;  // tiles; bit s: stage s loaded, bit 16 + s: parity of its last load
      bool ok = true;
      int gi = sh.first;
      Group g = p.groups[gi];
      for (long long at = c0; ok && at < c1;) {
        const Segment seg = segment_of(g, c0, c1, blockIdx.x);
        at = g.tile0 + seg.j1;
        const Pages pg = group_pages(g.pos0, g.npos, p.W, p.m, p.log_bs, p.comp.table != nullptr);
        Group gn = g;
        if (at < c1) gn = p.groups[gi + 1];
        for (int jb = seg.j0; ok && jb < seg.j1; jb += batch) {
          const int v = jb * ppt + lane;
          PageMeta pm = {0, 2, 0.f, 0.f};
          int id = -1;
          bool good = false;
          if (v < pg.nraw + pg.ncomp && v < seg.j1 * ppt) {
            const bool comp = v >= pg.nraw;
            const CacheSet &cs = comp ? p.comp : p.raw;
            const int page = comp ? v - pg.nraw : pg.rp0 + v;
            id = cs.table[(size_t)g.r * cs.cols + page % cs.cols];
            pm.kind = comp;
            pm.key0 = page << p.log_bs;
            pm.scale = __int_as_float(0x7fc00000);
            good = id >= 0 && id < cs.nblocks;
            if (good) pm.scale = cs.scale[id];
            else atomicExch(status, HCA_ERR_CACHE);
          }
          const uint32_t have = __ballot_sync(0xffffffffu, good);
          const int jn = min(batch, seg.j1 - jb);
          for (int k = 0; k < jn; ++k, ++n) {
            const int st = n % C::kStages;
            if (n >= (uint32_t)C::kStages)
              ok = wait_warp(&sh.kv_empty[st], ((n / C::kStages) - 1) & 1, abort_flag, status, p.wait_ns);
            if (!ok) break;
            const uint32_t mine = (have >> (k * ppt)) & ((1u << ppt) - 1u);
            if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[st], __popc(mine) * page_bytes);
            issued = (issued | (1u << st)) & ~(1u << (16 + st));
            issued |= ((n / C::kStages) & 1u) << (16 + st);
            __syncwarp();
            if (lane / ppt == k) {
              const int slot = lane % ppt;
              uint8_t *dst = smem + st * C::kStageBytes + slot * page_bytes;
              if (good && pm.kind) tma_load_2d(&map_comp, &sh.kv_full[st], dst, 0, id << p.log_bs);
              else if (good) tma_load_2d(&map_raw, &sh.kv_full[st], dst, 0, id << p.log_bs);
              pm.log2_scale = log2f(pm.scale);
              sh.meta[st][slot] = pm;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.kv_full[st]);
          }
        }
        g = gn;
        ++gi;
      }
      if (!ok && lane == 0) {
        volatile int never = 0;
        for (int s = 0; s < C::kStages; ++s)
          if (issued & (1u << s)) mbar_wait(&sh.kv_full[s], (issued >> (16 + s)) & 1u, &never, status, 100000000ull);
      }
      __syncwarp();
    }
  } else if (warp == C::kSoft / 32 + 1) {
    // -------------------------------------------------------------- MMA
    if (busy) {
      const uint32_t kv0 = smem_u32(smem), q0 = smem_u32(smem + C::kOffQ), p0 = smem_u32(smem + C::kOffP);
      uint64_t dk, dv, dq;
      if constexpr (D == 128) {
        dk = smem_desc_sw128(kv0, 16, 1024);
        dv = smem_desc_sw128(kv0, 16, 1024);
        dq = smem_desc_sw128(q0, 16, 1024);
      } else {
        // K^T has 64 rows: M = 128 takes them twice (leading offset 0), the
        // upper half of O's lanes is not read
        dk = smem_desc_sw64(kv0, 16, 512);
        dv = smem_desc_sw64(kv0, 0, 512);
        dq = smem_desc_sw64(q0, 16, 512);
      }
      const uint64_t dp = smem_desc_sw128(p0, 16, 1024);
      const uint32_t id_s = idesc_e4m3_f32(128, NQ, false, false);
      const uint32_t id_o = idesc_e4m3_f32(128, NQ == 128 ? 128 : 2 * NQ, true, true);
      uint32_t n = 0, nseg = 0;
      bool ok = true, issued = false, prev_first = false;
      if (p.stall) {
        injected_stall(&sh.never, abort_flag, status, p.wait_ns);
        ok = false;
      }
      // O (+)= K^T P of tile k
      auto issue_pv = [&](uint32_t k, bool fresh) {
        if (!wait_warp(&sh.p_full[k & 1], (k >> 1) & 1, abort_flag, status, p.wait_ns)) return false;
        tc_fence_after();
        const uint32_t st = k % C::kStages;
        const uint64_t a = dv + desc_bytes(st * C::kStageBytes), b = dp + desc_bytes((k & 1) * C::kPBytes);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            mma_f8_ss(tmem + 2 * NQ, a + desc_bytes(kk * 32 * D), b + desc_bytes(kk * 4096), id_o, !fresh || kk > 0);
            if constexpr (NQ == 128)
              mma_f8_ss(tmem + 3 * NQ, a + desc_bytes(kk * 32 * D), b + desc_bytes(C::kPHalf + kk * 4096), id_o,
                        !fresh || kk > 0);
          }
          mma_commit(&sh.pv_done[k & 1]);
          mma_commit(&sh.kv_empty[st]);
        }
        __syncwarp();
        return true;
      };
      int gi = sh.first;
      Group g = p.groups[gi];
      for (long long at = c0; ok && at < c1; ++nseg) {
        const Segment seg = segment_of(g, c0, c1, blockIdx.x);
        at = g.tile0 + seg.j1;
        if (at < c1) g = p.groups[++gi];
        for (int j = seg.j0; ok && j < seg.j1; ++j, ++n) {
          const bool first = j == seg.j0;
          // a group's q is written after the last softmax of the group before
          if (first && n > 0) ok = issue_pv(n - 1, prev_first);
          const uint32_t st = n % C::kStages;
          if (ok) ok = wait_warp(&sh.kv_full[st], (n / C::kStages) & 1, abort_flag, status, p.wait_ns);
          if (ok && n >= 2) ok = wait_warp(&sh.s_free[n & 1], ((n >> 1) - 1) & 1, abort_flag, status, p.wait_ns);
          if (ok && first) ok = wait_warp(&sh.q_full, nseg & 1, abort_flag, status, p.wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = dk + desc_bytes(st * C::kStageBytes);
          if (elect_one()) {
#pragma unroll
            for (int hl = 0; hl < 2; ++hl)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_f8_ss(tmem + (n & 1) * NQ, a + desc_bytes(kk * 32), dq + desc_bytes(hl * NQ * D + kk * 32), id_s,
                          hl + kk > 0);
            mma_commit(&sh.s_full[n & 1]);
          }
          __syncwarp();
          issued = true;
          if (!first) ok = issue_pv(n - 1, prev_first);
          prev_first = first;
        }
      }
      if (ok && n > 0) ok = issue_pv(n - 1, prev_first);
      if (!ok && issued) {
        volatile int never = 0;
        if (elect_one()) mma_commit(&sh.drain);
        __syncwarp();
        if (lane == 0) mbar_wait(&sh.drain, 0, &never, status, 100000000ull);
        __syncwarp();
      }
    }
  } else if (ntiles < 0) {
    // the schedule was refused
    const size_t rows = (size_t)p.N * p.H;
    const uint4 nan4 = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
    for (size_t i = (size_t)blockIdx.x * C::kSoft + tid; i < rows * (D / 8); i += (size_t)gridDim.x * C::kSoft)
      reinterpret_cast<uint4 *>(p.out)[i] = nan4;
    for (size_t i = (size_t)blockIdx.x * C::kSoft + tid; i < rows; i += (size_t)gridDim.x * C::kSoft)
      p.lse[i] = __int_as_float(0x7fc00000);
  } else if (busy) {
    // ---------------------------------------------------------- softmax
    // A wait that gave up (abort) does not leave the loop: every thread goes
    // through all named barriers, later waits return at once.
    const int wg = warp >> 2, r = tid & 127;  // warpgroup; key of a tile, dimension of O
    const int col0 = wg * CW;
    const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t bar_wg = 1 + wg, bar_all = 3;
    auto wait = [&](uint64_t *bar, uint32_t parity) { (void)wait_warp(bar, parity, abort_flag, status, p.wait_ns); };

    // q of a group into shared memory; returns log2(e) * scale / (its factor)
    auto load_q = [&](const Group &g) {
      constexpr int kUnits = NQ * D / 16 / C::kSoft;  // 16 values each
      const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + ((size_t)g.row0 * p.H + g.slice * p.HS) * D;
      const int nreal = real_columns(p, g);
      uint4 u[kUnits > 0 ? kUnits : 1][2];
      constexpr int kAll = NQ * D / 16;
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < (kUnits > 0 ? kUnits : 1); ++k) {
        const int i = tid + k * C::kSoft, c = i / (D / 16);
        u[k][0] = u[k][1] = make_uint4(0, 0, 0, 0);
        if (i < kAll && c < nreal) {
          const uint4 *src = reinterpret_cast<const uint4 *>(q) + (size_t)i * 2;
          u[k][0] = src[0];
          u[k][1] = src[1];
        }
        const uint32_t w[8] = {u[k][0].x, u[k][0].y, u[k][0].z, u[k][0].w, u[k][1].x, u[k][1].y, u[k][1].z, u[k][1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = fabsf(__uint_as_float(w[e] << 16)), b = fabsf(__uint_as_float(w[e] & 0xffff0000u));
          if (a < INFINITY) amax = fmaxf(amax, a);
          if (b < INFINITY) amax = fmaxf(amax, b);
        }
      }
      const int wm = __reduce_max_sync(0xffffffffu, __float_as_int(amax));
      if (lane == 0) sh.amax[warp] = __int_as_float(wm);
      if (r < CW) sh.nref[col0 + r] = 0.f;
      named_bar_sync(bar_all, C::kSoft);
      amax = sh.amax[0];
#pragma unroll
      for (int w = 1; w < 4 * C::WG; ++w) amax = fmaxf(amax, sh.amax[w]);
      const float s = exp2_int(scale_exponent(amax)), inv = 1.f / s;
#pragma unroll
      for (int k = 0; k < (kUnits > 0 ? kUnits : 1); ++k) {
        const int i = tid + k * C::kSoft, c = i / (D / 16), ch = i % (D / 16);
        if (i >= kAll) break;
        const uint32_t w[8] = {u[k][0].x, u[k][0].y, u[k][0].z, u[k][0].w, u[k][1].x, u[k][1].y, u[k][1].z, u[k][1].w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = __uint_as_float(w[e] << 16), b = __uint_as_float(w[e] & 0xffff0000u);
          // an infinity becomes NaN, not 448
          const uint32_t h2 = f16x2_rn(fmaf(a, 0.f, a * inv), fmaf(b, 0.f, b * inv));
          uint32_t h, l;
          split2(h2, 0x3c003c00u, h, l);  // factor 1: one accumulator for both
          if (e & 1) {
            hi[e >> 1] |= h << 16;
            lo[e >> 1] |= l << 16;
          } else {
            hi[e >> 1] = h;
            lo[e >> 1] = l;
          }
        }
        const int off = D == 128 ? c * 128 + ((ch ^ (c & 7)) << 4) : c * 64 + ((ch ^ ((c >> 1) & 3)) << 4);
        *reinterpret_cast<uint4 *>(smem + C::kOffQ + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(smem + C::kOffQ + NQ * D + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_async_smem();
      mbar_arrive(&sh.q_full);
      return s * p.scale * 1.4426950408889634f;
    };

    uint32_t n = 0;
    int gi = sh.first;
    Group g = p.groups[gi];
    float cs = load_q(g);
    for (long long at = c0; at < c1;) {
      const Segment seg = segment_of(g, c0, c1, blockIdx.x);
      at = g.tile0 + seg.j1;
      Group gn = g;
      if (at < c1) gn = p.groups[++gi];
      const int nfull = g.npos * p.HS, nreal = real_columns(p, g);
      float l[CW];
#pragma unroll
      for (int c = 0; c < CW; ++c) l[c] = 0.f;
      bool unset = true;  // some column has seen no key yet
      for (int j = seg.j0; j < seg.j1; ++j, ++n) {
        const bool first = j == seg.j0;
        const uint32_t st = n % C::kStages, b = n & 1;
        wait(&sh.kv_full[st], (n / C::kStages) & 1);  // for the pages' data; the MMA warp has waited for the rows
        const PageMeta pm = sh.meta[st][r >> p.log_bs];
        int ca = 0, cb = 0;
        if (pm.kind < 2)
          key_columns(pm.kind == 1, (long long)pm.key0 + (r & ((1 << p.log_bs) - 1)), g.pos0, g.npos, p.HS, p.W, p.m, ca, cb);
        const bool none = cb <= ca;
        if (ca == 0 && cb == nfull) cb = NQ;  // columns that stand for nothing do no harm
        const bool full = __all_sync(0xffffffffu, ca == 0 && cb == NQ);
        const float ck = cs * pm.scale, inv_s = 1.f / pm.scale;
        wait(&sh.s_full[b], (n >> 1) & 1);
        tc_fence_after();
        uint32_t t[CW];
        load_cols<CW>(lane_addr + b * NQ + col0, t);
        tc_fence_before();
        mbar_arrive(&sh.s_free[b]);
        // t = log2(probability * scale) relative to the column's reference
        const uint64_t ck2 = f32x2(__float_as_uint(ck), __float_as_uint(ck));
        const uint64_t lb2 = f32x2(__float_as_uint(pm.log2_scale), __float_as_uint(pm.log2_scale));
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < CW; c += 4) {
          const float4 nr = *reinterpret_cast<const float4 *>(&sh.nref[col0 + c]);
          const uint64_t n01 = f32x2(__float_as_uint(nr.x), __float_as_uint(nr.y));
          const uint64_t n23 = f32x2(__float_as_uint(nr.z), __float_as_uint(nr.w));
          float a0, a1, a2, a3;
          f32x2_split(ffma2(f32x2(t[c], t[c + 1]), ck2, fadd2(n01, lb2)), a0, a1);
          f32x2_split(ffma2(f32x2(t[c + 2], t[c + 3]), ck2, fadd2(n23, lb2)), a2, a3);
          t[c] = __float_as_uint(a0);
          t[c + 1] = __float_as_uint(a1);
          t[c + 2] = __float_as_uint(a2);
          t[c + 3] = __float_as_uint(a3);
        }
        if (!full) {
#pragma unroll
          for (int c = 0; c < CW; ++c)
            if (col0 + c < ca || col0 + c >= cb) t[c] = 0xff800000u;
        }
        {
          float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < CW; c += 8)
#pragma unroll
            for (int q = 0; q < 4; ++q) m[q] = fmax3(m[q], __uint_as_float(t[c + 2 * q]), __uint_as_float(t[c + 2 * q + 1]));
          top = fmaxf(fmax3(m[0], m[1], m[2]), m[3]);
        }
        if (unset || named_bar_any(bar_wg, 128, top > kTopLog2)) {
          // the columns' maxima over the tile
#pragma unroll
          for (int h = 0; h < CW; h += 32) {
            int mine = 0;
#pragma unroll
            for (int y = 0; y < (CW < 32 ? CW : 32); ++y) {
              const int mx = __reduce_max_sync(0xffffffffu, ordered(__uint_as_float(t[h + y])));
              if (lane == y) mine = mx;
            }
            if (h + lane < CW) sh.wmax[warp][h + lane] = mine;
          }
          named_bar_sync(bar_wg, 128);
          bool un = false;
          if (r < CW) {
            const int w0 = 4 * wg;
            const float mx = unordered(max(max(sh.wmax[w0][r], sh.wmax[w0 + 1][r]), max(sh.wmax[w0 + 2][r], sh.wmax[w0 + 3][r])));
            un = first ? col0 + r < nreal : sh.unset[col0 + r] != 0;
            float d = 0.f, f = 1.f;
            if (un) {
              if (!(mx == -INFINITY)) {
                un = false;
                if (mx == mx) d = mx - kRefLog2;
              }
            } else if (mx > kRefLog2) {
              d = mx - kRefLog2;
              f = ex2_approx(-d);
            }
            sh.delta[col0 + r] = d;
            sh.fac[col0 + r] = f;
            sh.nref[col0 + r] -= d;
            sh.unset[col0 + r] = un;
          }
          unset = named_bar_any(bar_wg, 128, un);
#pragma unroll
          for (int c = 0; c < CW; ++c) {
            t[c] = __float_as_uint(__uint_as_float(t[c]) - sh.delta[col0 + c]);
            l[c] *= sh.fac[col0 + c];
          }
          if (!first) {
            wait(&sh.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < CW; c += 16) {
#pragma unroll
              for (int hl = 0; hl < 2; ++hl) {
                uint32_t o[16];
                tmem_ld16(lane_addr + (2 + hl) * NQ + col0 + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * sh.fac[col0 + c + y]);
                tmem_st16(lane_addr + (2 + hl) * NQ + col0 + c, o);
              }
            }
            tmem_wait_st();
          }
        }
        // probabilities, the row sums, and two e4m3 numbers for each
        if (n >= 2) wait(&sh.pv_done[b], ((n >> 1) - 1) & 1);  // P's buffer is free
        uint8_t *prow = smem + C::kOffP + b * C::kPBytes + r * 128;
        const uint64_t inv2 = f32x2(__float_as_uint(inv_s), __float_as_uint(inv_s));
#pragma unroll
        for (int c = 0; c < CW; c += 16) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int y = 0; y < 16; y += 2) {
            const float e0 = ex2_approx(__uint_as_float(t[c + y])), e1 = ex2_approx(__uint_as_float(t[c + y + 1]));
            uint64_t l2 = f32x2(__float_as_uint(l[c + y]), __float_as_uint(l[c + y + 1]));
            // a masked key's scale may be anything
            l2 = none ? l2 : ffma2(f32x2(__float_as_uint(e0), __float_as_uint(e1)), inv2, l2);
            f32x2_split(l2, l[c + y], l[c + y + 1]);
            uint32_t h, lw;
            split2(f16x2_rn(e0, e1), 0x50005000u, h, lw);  // 2^5
            if (y & 2) {
              hi[y >> 2] |= h << 16;
              lo[y >> 2] |= lw << 16;
            } else {
              hi[y >> 2] = h;
              lo[y >> 2] = lw;
            }
          }
          const int ch = (col0 + c) >> 4;
          if constexpr (NQ == 128) {
            *reinterpret_cast<uint4 *>(prow + ((ch ^ (r & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(prow + C::kPHalf + ((ch ^ (r & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          } else {
            *reinterpret_cast<uint4 *>(prow + ((ch ^ (r & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(prow + (((NQ / 16 + ch) ^ (r & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        if (wg == 0 && !full) {
          uint4 *row = reinterpret_cast<uint4 *>(smem + st * C::kStageBytes + r * D);
          bool clear = none || pm.scale != pm.scale;
          if (!clear && cb - ca < NQ) {
            // seen by some columns only: NaN in it is their affair
            uint32_t nan = 0;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) nan |= nan_bytes(row[c]);
            clear = nan != 0;
          }
          if (clear) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) row[c] = make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(&sh.p_full[b]);
      }
      // the next group's q: every product with this one's has been made
      const float nref = r < CW ? sh.nref[col0 + r] : 0.f;
      if (at < c1) cs = load_q(gn);
      // sums over the keys
      if constexpr (CW >= 32) {
#pragma unroll
        for (int h = 0; h < CW; h += 32) sh.lred[warp][h + lane] = column_sum<32>(*reinterpret_cast<float(*)[32]>(&l[h]), lane);
      } else {
        const float s = column_sum<CW>(l, lane);
        if (lane < CW) sh.lred[warp][lane] = s;
      }
      named_bar_sync(bar_wg, 128);
      const size_t row0 = (size_t)g.row0 * p.H + g.slice * p.HS;  // row of column 0: columns are rows of q and out in order
      if (r < CW) {
        const int w0 = 4 * wg, c = col0 + r;
        float s = (sh.lred[w0][r] + sh.lred[w0 + 1][r]) + (sh.lred[w0 + 2][r] + sh.lred[w0 + 3][r]);
        if (*abort_flag) s = __int_as_float(0x7fc00000);
        if (c < nreal) {
          if (seg.whole) p.lse[row0 + c] = (log2f(s) - nref) * 0.69314718055994531f;
          else p.part_ml[(size_t)seg.slot * NQ + c] = make_float2(-nref, s);
        }
        sh.inv[c] = seg.whole ? 1.f / s : 1.f;
      }
      named_bar_sync(bar_wg, 128);
      wait(&sh.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
      tc_fence_after();
      if ((warp & 3) * 32 < D) {
#pragma unroll 1
        for (int c = 0; c < CW; c += 16) {
          uint32_t hi[16], lo[16];
          tmem_ld16(lane_addr + 2 * NQ + col0 + c, hi);
          tmem_ld16(lane_addr + 3 * NQ + col0 + c, lo);
          tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            const int cc = col0 + c + y;
            const float o = fmaf(__uint_as_float(lo[y]), 1.f / 32.f, __uint_as_float(hi[y])) * sh.inv[cc];
            if (cc < nreal) {
              if (seg.whole) static_cast<__nv_bfloat16 *>(p.out)[(row0 + cc) * D + r] = __float2bfloat16_rn(o);
              else p.part_o[((size_t)seg.slot * NQ + cc) * D + r] = o;
            }
          }
        }
      }
      tc_fence_before();
      g = gn;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// Map of a pool's rows: {D, rows} bytes, boxes of one block, swizzled by rows.
bool make_pool_map(CUtensorMap *m, const CacheSet &s, int D, int bs) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)s.nblocks * bs};
  cuuint64_t strides[1] = {(cuuint64_t)D};
  cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)bs};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(s.pool), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NQ, int D>
cudaError_t launch(const AttnParams &p, const CUtensorMap &raw, const CUtensorMap &comp, cudaStream_t st) {
  using C = Cfg<NQ, D>;
  static SmemAttrOnce attr;
  const cudaError_t e = attr.ensure(reinterpret_cast<const void *>(hca_cache_attn_kernel<NQ, D>), C::kSmem);
  if (e != cudaSuccess) return e;
  ProfScope prof(kKCacheAttn, st);
  hca_cache_attn_kernel<NQ, D><<<p.grid, C::kThreads, C::kSmem, st>>>(raw, comp, p);
  return cudaGetLastError();
}

}  // namespace

namespace cache {

int tc_cache_ctas(int NQ) { return NQ == 128 ? 1 : 2; }

cudaError_t tc_cache_attn(const AttnParams &p, cudaStream_t st) {
  CUtensorMap raw, comp;
  // without blocks there is nothing to load: every id is out of range
  const int bs = 1 << p.log_bs;
  if (p.raw.nblocks > 0 && !make_pool_map(&raw, p.raw, p.D, bs)) return cudaErrorInvalidValue;
  const bool has = p.comp.table && p.comp.nblocks > 0;
  if (has && !make_pool_map(&comp, p.comp, p.D, bs)) return cudaErrorInvalidValue;
  if (p.raw.nblocks == 0) raw = has ? comp : CUtensorMap{};
  if (!has) comp = raw;
  const int which = (p.NQ == 16 ? 0 : p.NQ == 32 ? 1 : p.NQ == 64 ? 2 : 3) + (p.D == 64 ? 4 : 0);
  switch (which) {
    case 0: return launch<16, 128>(p, raw, comp, st);
    case 1: return launch<32, 128>(p, raw, comp, st);
    case 2: return launch<64, 128>(p, raw, comp, st);
    case 3: return launch<128, 128>(p, raw, comp, st);
    case 4: return launch<16, 64>(p, raw, comp, st);
    case 5: return launch<32, 64>(p, raw, comp, st);
    case 6: return launch<64, 64>(p, raw, comp, st);
    default: return launch<128, 64>(p, raw, comp, st);
  }
}

}  // namespace cache
}  // namespace hca
