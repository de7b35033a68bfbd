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
  static constexpr int WG = NQ == 128 ? 2 : 1;    // softmax warpgroups, CW columns each
  static constexpr int CW = NQ / WG;
  static constexpr int kSoft = 128 * WG;          // softmax threads
  static constexpr int kThreads = kSoft + 128;    // and the warpgroup of the TMA and the MMA warp
  static constexpr int kCtas = NQ == 128 ? 1 : 2; // CTAs per SM
  // Registers.  A softmax thread holds CW scores and CW sums, more than an even
  // share of the SM's registers allows: the other warpgroup gives up some of its.
  static constexpr int kRegsSoft = NQ == 128 ? 216 : 192, kRegsIssue = 64;
  static constexpr int kRegsLaunch = NQ == 128 ? 168 : 128;
  static_assert(kSoft * kRegsSoft + 128 * kRegsIssue <= kThreads * kRegsLaunch, "register split must fit the launch");
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

// A page of a tile.
enum PageKind { kRaw = 0, kComp = 1, kNoPage = 2, kAllSeen = 3 };  // kAllSeen: every column sees every key
struct __align__(16) PageMeta {
  int key0_kind;  // first key (a multiple of 16) + kind
  float scale, log2_scale, inv_scale;
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
  // the CTA's pieces of groups, in order (more than there is room for: read
  // from the schedule kernel's groups)
  Segment seg[C::kThreads];
  int gbase[C::kThreads];
  long long scan[33];
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

__device__ __forceinline__ void st_shared(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// Four values to two e4m3 numbers each: hi = e4m3(v), lo = e4m3((v - hi) * f).
// fp16 holds v to 11 bits, hi and the difference exactly.
__device__ __forceinline__ void split4(float v0, float v1, float v2, float v3, uint32_t f2, uint32_t &hi, uint32_t &lo) {
  asm("{\n\t.reg .b32 a, b, c, d;\n\t.reg .b16 x, y;\n\t"
      "cvt.rn.f16x2.f32 a, %3, %2;\n\t"
      "cvt.rn.f16x2.f32 b, %5, %4;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 x, a;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 y, b;\n\t"
      "mov.b32 %0, {x, y};\n\t"
      "cvt.rn.f16x2.e4m3x2 c, x;\n\t"
      "cvt.rn.f16x2.e4m3x2 d, y;\n\t"
      "sub.rn.f16x2 a, a, c;\n\t"
      "sub.rn.f16x2 b, b, d;\n\t"
      "mul.rn.f16x2 a, a, %6;\n\t"
      "mul.rn.f16x2 b, b, %6;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 x, a;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 y, b;\n\t"
      "mov.b32 %1, {x, y};\n\t}"
      : "=&r"(hi), "=r"(lo)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3), "r"(f2));
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
  int32_t *status = &p.err[blockIdx.x];

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
  if (warp == C::kSoft / 32 + 2) {
    tmem_alloc(&sh.tmem_base, C::kTmem);
    tmem_relinquish();
  }
  // the CTA's range of the line, and its pieces of groups
  long long ntiles, quota, c0, c1;
  if (p.in_cta) {
    // one thread per request, then one per group
    long long n = 0, all;
    bool ok = true;
    if (tid < p.R) ok = request_chunks(p, tid, n);
    const long long before = block_scan(n, sh.scan, all);
    if (tid < p.R) sh.gbase[tid] = (int)before;
    ok = __syncthreads_and(ok);
    Group g;
    g.ntiles = 0;
    const bool mine = ok && tid < all;
    if (mine) {
      int lo = 0, hi = p.R;  // gbase[lo] <= tid < gbase[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.gbase[mid] <= tid) lo = mid; else hi = mid;
      }
      ok = chunk_group(p, lo, tid - sh.gbase[lo], g);
    }
    g.tile0 = block_scan(g.ntiles, sh.scan, ntiles);
    if (!__syncthreads_and(ok)) ntiles = -1;
    quota = cta_quota(ntiles, p.grid, p.min_tiles);
    c0 = quota * blockIdx.x;
    c1 = min(c0 + quota, ntiles);
    const bool in = mine && g.tile0 < c1 && g.tile0 + g.ntiles > c0;
    if (in && g.tile0 <= c0) sh.first = tid;
    __syncthreads();
    if (in) {
      const Segment x = segment_of(g, c0, c1, blockIdx.x);
      sh.seg[tid - sh.first] = x;
      if (x.last()) p.border[blockIdx.x] = border_of(p, g, c0, c1, quota, blockIdx.x);
    }
  } else {
    ntiles = p.hdr->ntiles;
    quota = cta_quota(ntiles, p.grid, p.min_tiles);
    c0 = quota * blockIdx.x;
    c1 = min(c0 + quota, ntiles);
    if (c0 < c1) {
      const int ng = p.hdr->ngroups;
      if (warp == 0) {
        const int g = find_group(p.groups, ng, c0);
        if (lane == 0) sh.first = g;
      } else if (warp == 1) {
        const int g = find_group(p.groups, ng, c1 - 1);
        if (lane == 0) p.border[blockIdx.x] = border_of(p, p.groups[g], c0, c1, quota, blockIdx.x);
      }
      __syncthreads();
      const int gi = sh.first + tid;
      if (gi < ng) {
        const Group g = p.groups[gi];
        if (g.tile0 < c1) sh.seg[tid] = segment_of(g, c0, c1, blockIdx.x);
      }
    }
  }
  const bool busy = c0 < c1;
  if (tid == 0) {
    p.err[blockIdx.x] = ntiles < 0 ? HCA_ERR_CACHE : HCA_OK;
    if (!busy) p.border[blockIdx.x] = Border{0, 0, 0, 0};
  }
  auto segment = [&](int k) { return k < C::kThreads ? sh.seg[k] : segment_of(p.groups[sh.first + k], c0, c1, blockIdx.x); };
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  if (warp >= C::kSoft / 32) {
  setmaxnreg_dec<C::kRegsIssue>();
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
      for (int k = 0; ok; ++k) {
        const Segment g = segment(k);
        const Pages pg = group_pages(g.pos0, g.npos, p.W, p.m, p.log_bs, p.comp.table != nullptr);
        for (int jb = g.j0; ok && jb < g.j1; jb += batch) {
          const int v = jb * ppt + lane;
          PageMeta pm = {kNoPage, 1.f, 0.f, 0.f};
          int id = -1;
          bool good = false, comp = false;
          if (v < pg.nraw + pg.ncomp && v < g.j1 * ppt) {
            comp = v >= pg.nraw;
            const CacheSet &cs = comp ? p.comp : p.raw;
            const int page = comp ? v - pg.nraw : pg.rp0 + v;
            id = cs.table[(size_t)g.r * cs.cols + page % cs.cols];
            const int key0 = page << p.log_bs;
            const long long end = (long long)key0 + (1 << p.log_bs);
            const bool all = comp ? end * p.m <= g.pos0 + 1 : end <= (long long)g.pos0 + 1 && key0 > g.pos0 + g.npos - 1 - p.W;
            pm.key0_kind = key0 + (all ? kAllSeen : comp ? kComp : kRaw);
            pm.scale = __int_as_float(0x7fc00000);
            good = id >= 0 && id < cs.nblocks;
            if (good) pm.scale = cs.scale[id];
            else atomicExch(status, HCA_ERR_CACHE);
          }
          const uint32_t have = __ballot_sync(0xffffffffu, good);
          const int jn = min(batch, g.j1 - jb);
          for (int t = 0; t < jn; ++t, ++n) {
            const int st = n % C::kStages;
            if (n >= (uint32_t)C::kStages)
              ok = wait_warp(&sh.kv_empty[st], ((n / C::kStages) - 1) & 1, abort_flag, status, p.wait_ns);
            if (!ok) break;
            const uint32_t mine = (have >> (t * ppt)) & ((1u << ppt) - 1u);
            if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[st], __popc(mine) * page_bytes);
            issued = (issued | (1u << st)) & ~(1u << (16 + st));
            issued |= ((n / C::kStages) & 1u) << (16 + st);
            __syncwarp();
            if (lane / ppt == t) {
              const int slot = lane % ppt;
              uint8_t *dst = smem + st * C::kStageBytes + slot * page_bytes;
              if (good && comp) tma_load_2d(&map_comp, &sh.kv_full[st], dst, 0, id << p.log_bs);
              else if (good) tma_load_2d(&map_raw, &sh.kv_full[st], dst, 0, id << p.log_bs);
              if (pm.key0_kind != kNoPage) {
                pm.log2_scale = log2f(pm.scale);
                pm.inv_scale = 1.f / pm.scale;
              }
              sh.meta[st][slot] = pm;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.kv_full[st]);
          }
        }
        if (g.last()) break;
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
    // S of tile n + 1 is issued before O of tile n, so that it is there when the
    // softmax of tile n ends.  Products run in the order of issue: S of tile n
    // complete means O of tile n - 2 complete, whose P buffer tile n takes.
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
      for (; ok; ++nseg) {
        const Segment seg = segment(nseg);
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
        if (seg.last()) break;
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
  }
  } else {
  setmaxnreg_inc<C::kRegsSoft>();
  if (ntiles < 0) {
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
    const uint32_t bar_wg = 1 + wg, bar_all = 1 + C::WG;
    auto wait = [&](uint64_t *bar, uint32_t parity) { (void)wait_warp(bar, parity, abort_flag, status, p.wait_ns); };

    // q of a group into shared memory; returns log2(e) * scale / (its factor)
    auto load_q = [&](const Segment &g) {
      constexpr int kUnits = NQ * D / 16 / C::kSoft;  // 16 values each
      const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + ((size_t)g.row0 * p.H + g.slice() * p.HS) * D;
      const int nreal = real_columns(p, g.npos, g.slice());
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
        for (int e = 0; e < 4; ++e) {
          float v[4] = {__uint_as_float(w[2 * e] << 16), __uint_as_float(w[2 * e] & 0xffff0000u),
                        __uint_as_float(w[2 * e + 1] << 16), __uint_as_float(w[2 * e + 1] & 0xffff0000u)};
#pragma unroll
          for (int x = 0; x < 4; ++x) v[x] = fmaf(v[x], 0.f, v[x] * inv);  // an infinity becomes NaN, not 448
          split4(v[0], v[1], v[2], v[3], 0x3c003c00u, hi[e], lo[e]);        // factor 1: one accumulator for both
        }
        const int off = D == 128 ? c * 128 + ((ch ^ (c & 7)) << 4) : c * 64 + ((ch ^ ((c >> 1) & 3)) << 4);
        st_shared(smem_u32(smem) + C::kOffQ + off, hi);
        st_shared(smem_u32(smem) + C::kOffQ + NQ * D + off, lo);
      }
      fence_async_smem();
      mbar_arrive(&sh.q_full);
      return s * p.scale * 1.4426950408889634f;
    };

    uint32_t n = 0;
    float cs = load_q(segment(0));
    for (int k = 0;; ++k) {
      const Segment g = segment(k);
      const int nreal = real_columns(p, g.npos, g.slice());
      float l[CW];
#pragma unroll
      for (int c = 0; c < CW; ++c) l[c] = 0.f;
      bool unset = true;  // some column has seen no key yet
      for (int j = g.j0; j < g.j1; ++j, ++n) {
        const bool first = j == g.j0;
        const uint32_t st = n % C::kStages, b = n & 1;
        wait(&sh.kv_full[st], (n / C::kStages) & 1);  // for the pages' data; the MMA warp has waited for the rows
        const PageMeta pm = sh.meta[st][r >> p.log_bs];
        const int kind = pm.key0_kind & 3;
        int ca = 0, cb = kind == kAllSeen ? NQ : 0;
        if (kind < kNoPage) {
          key_columns(kind == kComp, (long long)(pm.key0_kind & ~3) + (r & ((1 << p.log_bs) - 1)), g.pos0, g.npos, p.HS, p.W,
                      p.m, ca, cb);
          if (ca == 0 && cb == g.npos * p.HS) cb = NQ;  // columns that stand for nothing do no harm
        }
        const bool none = cb <= ca;
        const bool full = __all_sync(0xffffffffu, ca == 0 && cb == NQ);
        const float ck = cs * pm.scale;
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
        const uint32_t prow = smem_u32(smem) + C::kOffP + b * C::kPBytes + r * 128;
        const uint64_t inv2 = f32x2(__float_as_uint(pm.inv_scale), __float_as_uint(pm.inv_scale));
#pragma unroll
        for (int c = 0; c < CW; c += 16) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int y = 0; y < 16; y += 4) {
            float e[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) e[x] = ex2_approx(__uint_as_float(t[c + y + x]));
#pragma unroll
            for (int x = 0; x < 4; x += 2) {
              const uint64_t l2 = f32x2(__float_as_uint(l[c + y + x]), __float_as_uint(l[c + y + x + 1]));
              f32x2_split(ffma2(f32x2(__float_as_uint(e[x]), __float_as_uint(e[x + 1])), inv2, l2), l[c + y + x],
                          l[c + y + x + 1]);
            }
            split4(e[0], e[1], e[2], e[3], 0x50005000u, hi[y >> 2], lo[y >> 2]);  // 2^5
          }
          const int ch = (col0 + c) >> 4;
          constexpr int kLo = NQ == 128 ? 0 : NQ / 16;  // P_lo's first 16-byte chunk
          st_shared(prow + ((ch ^ (r & 7)) << 4), hi);
          st_shared(prow + C::kPHalf + (((kLo + ch) ^ (r & 7)) << 4), lo);
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
      if (!g.last()) cs = load_q(segment(k + 1));
      // sums over the keys
      if constexpr (CW >= 32) {
#pragma unroll
        for (int h = 0; h < CW; h += 32) sh.lred[warp][h + lane] = column_sum<32>(*reinterpret_cast<float(*)[32]>(&l[h]), lane);
      } else {
        const float s = column_sum<CW>(l, lane);
        if (lane < CW) sh.lred[warp][lane] = s;
      }
      named_bar_sync(bar_wg, 128);
      const bool whole = g.slot < 0;
      const size_t row0 = (size_t)g.row0 * p.H + g.slice() * p.HS;  // row of column 0: columns are rows of q and out in order
      if (r < CW) {
        const int w0 = 4 * wg, c = col0 + r;
        float s = (sh.lred[w0][r] + sh.lred[w0 + 1][r]) + (sh.lred[w0 + 2][r] + sh.lred[w0 + 3][r]);
        if (*abort_flag) s = __int_as_float(0x7fc00000);
        if (c < nreal) {
          if (whole) p.lse[row0 + c] = (log2f(s) - nref) * 0.69314718055994531f;
          else p.part_ml[(size_t)g.slot * NQ + c] = make_float2(-nref, s);
        }
        sh.inv[c] = whole ? 1.f / s : 1.f;
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
              if (whole) static_cast<__nv_bfloat16 *>(p.out)[(row0 + cc) * D + r] = __float2bfloat16_rn(o);
              else p.part_o[((size_t)g.slot * NQ + cc) * D + r] = o;
            }
          }
        }
      }
      tc_fence_before();
      if (g.last()) break;
    }
  }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kSoft / 32 + 2) {
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
int tc_cache_threads(int NQ) {
  return NQ == 16 ? Cfg<16, 128>::kThreads : NQ == 32 ? Cfg<32, 128>::kThreads : NQ == 64 ? Cfg<64, 128>::kThreads
                                                                                       : Cfg<128, 128>::kThreads;
}

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
