// cross_bwd_tc.cuh -- gradients of cross attention on the 5th-generation tensor cores (bf16).
//
//   p_ij = exp(s_ij - lse_i),  D_i = dO_i . O_i,  ds_ij = p_ij (dO_i . v_j - D_i)
//   dQ_i = scale sum_j ds_ij k_j,  dK_j = scale sum_i ds_ij q_i,  dV_j = sum_i p_ij dO_i
//
// D_i comes from a kernel of its own (one pass over O and dO, 5.2 TB/s; inside dq_kernel its code and
// its loads held up the other warps).  Two more, so that every sum has one owner and a fixed order (no
// atomics): dq_kernel keeps a query tile and walks the keys, dkv_kernel keeps a key tile and walks the
// queries.  Each forms the scores and dP = dO V^T again (7 products of a tile pair instead of 5).  p
// and ds go back to tensor memory as bf16 (rounded once each, for the product that follows); the
// softmax scale is applied to the fp32 sums at the end.
//
// 32 heads of 75600 queries and 300 keys (929 GFLOP in 5 products) at 1965 MHz: 1588 us with D's pass of 227,
// which is 585 TFLOP/s, or 819 for the 7 products.  What bounds it is the chain of a step, score product ->
// exponentials -> dP -> ds -> product, of which tensor memory holds one and a half steps; the third key
// tile of 44 keys costs dkv_kernel as much as a full one.
//
// dq_kernel, tensor memory: S of even and odd steps [0, 256), dP [256, 384), dQ [384, 512); ds
// overwrites its S.  S of the next step and dP of the next step are computed while the math warps
// work on this one.
// dkv_kernel, scores transposed (keys are the rows): S^T [0, 128), dP^T [128, 256), dV [256, 384),
// dK [384, 512); p overwrites S^T, ds overwrites dP^T.  dV of this step and S^T of the next run while
// the math warps form ds, dK and the next dP^T while they form the next p.
//
// Warps: 0-15 math (thread = row; warps 4 c .. 4 c + 3 have columns [32 c, 32 c + 32) of a tile: with
// half as many, and twice the columns each, their latencies showed: a step took 2400 cycles for 1024
// of exponentials);
// 16-19 dq: dQ to memory; dkv: lse and D of the query tiles to come;
// 20 TMA producer; 21, 22 MMA issuers.  One CTA per SM, persistent.  Every wait is bounded.
//
// A wait on a barrier's parity tells its phase from the one before only, so no barrier may complete two
// phases ahead of anyone who waits for it.  Tiles and rings: a slot is filled again after everyone who
// waits for it has given it back (dkv: both issuers).  S, dP, dQ and the sums: the next phase is issued
// after all math (or storing) warps have arrived behind their wait.  p, ds, dpfree, dqfree, accfree:
// the next phase follows a product that the waiting issuer itself issues after its wait.  S^T of
// dkv_kernel, for which the other issuer waits too: see sfull.
#pragma once
#include "cross_tc.cuh"

namespace la {
namespace xb {

using xt::BM;
using xt::BN;
using xt::HALF;
using xt::LOG2E;
using xt::regs_dec;
using xt::regs_inc;
using xt::store32;
using xt::store_row32;

constexpr int THREADS = 768, MATH_WARPS = 16, AUX = 16, CTRL = 20;  // first auxiliary and control warp
constexpr uint32_t REGS_LAUNCH = 80, REGS_MATH = 88, REGS_AUX = 72, REGS_CTRL = 56;
static_assert(512 * REGS_MATH + 128 * REGS_AUX + 128 * REGS_CTRL <= THREADS * REGS_LAUNCH, "register split");

struct Args {
  int64_t B, H, Hkv, Nq, Nk, rows, keys;
  int64_t total;          // work items
  int32_t tiles;          // dq: query tiles per head; dkv: key tiles per head
  int32_t q_tiles;        // query tiles per head
  int32_t group;
  int32_t splits, per;    // dq: parts of the keys; dkv: parts of the group's query tiles
  FastDiv fd_tiles, fd_splits, fd_heads;  // tiles, splits, H (dq) or Hkv (dkv)
  float c, scale;         // scale * log2(e), scale
  const int32_t* count;
  xs::Str dq;
};

// ------------------------------------------------------------------------------------ dQ
template <int DP>
struct CfgQ {
  static constexpr uint32_t TILE = (DP / 64) * HALF;
  // Q and dO tiles of this item and the next (from HBM); K and V come from L2, and dP of the next step
  // leaves a V tile the time of a step's math to arrive in.
  static constexpr int QST = 4;
  static constexpr int KST = DP == 128 ? 2 : 4;
  static constexpr int VST = DP == 128 ? 1 : 4;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = QST * TILE;
  static constexpr uint32_t OFF_V = OFF_K + KST * TILE;
  static constexpr uint32_t OFF_BAR = OFF_V + VST * TILE;
  static constexpr uint32_t SMEM = OFF_BAR + 512 + 1024;
};
static_assert(CfgQ<128>::SMEM <= 232448 && CfgQ<64>::SMEM <= 232448, "shared memory budget");

template <int DP>
struct BarsQ {
  uint64_t qfull[CfgQ<DP>::QST], qempty[CfgQ<DP>::QST];
  uint64_t kfull[CfgQ<DP>::KST], kempty[CfgQ<DP>::KST];
  uint64_t vfull[CfgQ<DP>::VST], vempty[CfgQ<DP>::VST];
  uint64_t sfull[2], dsready[2];
  uint64_t dpfull, dpfree, dqfull, dqfree, final_[2];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(BarsQ<64>) <= 512, "barrier block too large");

constexpr uint32_t Q_S = 0, Q_DP = 256, Q_DQ = 384;

struct WorkQ {
  int64_t i;
  int32_t b, h, qt, split;
  int32_t k0, nk, keys;
};
__device__ __forceinline__ WorkQ get_q(const Args& a, int64_t i) {
  WorkQ w;
  w.i = i;
  uint32_t r = static_cast<uint32_t>(i);
  const uint32_t q = fdiv(r, a.fd_tiles);
  w.qt = static_cast<int32_t>(r - q * a.tiles);
  r = fdiv(q, a.fd_splits);
  w.split = static_cast<int32_t>(q - r * a.splits);
  w.b = static_cast<int32_t>(fdiv(r, a.fd_heads));
  w.h = static_cast<int32_t>(r - w.b * static_cast<uint32_t>(a.H));
  w.keys = a.count ? __ldg(a.count + w.b) : static_cast<int32_t>(a.Nk);
  w.k0 = w.split * a.per;
  const int32_t tiles = (w.keys + BN - 1) / BN - w.k0;
  w.nk = tiles < a.per ? tiles : a.per;
  if (w.nk < 0) w.nk = 0;
  return w;
}
// The item before this CTA's first, and the next one with work.
__device__ __forceinline__ WorkQ before_first_q() {
  WorkQ w;
  w.i = int64_t(blockIdx.x) - gridDim.x;
  w.nk = 0;
  return w;
}
__device__ __forceinline__ WorkQ next_q(const Args& a, WorkQ w) {
#pragma unroll 1
  do {
    w.i += gridDim.x;
    if (w.i >= a.total) break;
    w = get_q(a, w.i);
  } while (w.nk == 0);
  return w;
}
__device__ __forceinline__ int keys_of(const WorkQ& w, int j) {
  const int left = w.keys - (w.k0 + j) * BN;
  return left < BN ? left : BN;
}

template <int DP>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* m, int32_t n, int32_t h, int32_t b, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, (DP / 64) * HALF);
  tma_load_4d(dst, m, 0, n, h, b, bar);
  if (DP == 128) tma_load_4d(dst + HALF, m, 64, n, h, b, bar);
}

// Drains the copies of a ring that were issued and may still be in flight.
__device__ __forceinline__ void drain(uint64_t* full, uint32_t stages, uint32_t issued) {
  for (uint32_t j = issued > stages ? issued - stages : 0; j < issued; ++j)
    mbar_wait_drain(&full[j % stages], (j / stages) & 1);
}

template <int DP, int D>
__global__ void __launch_bounds__(THREADS, 1)
dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
          const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
          const __grid_constant__ Args a, const float* __restrict__ lse, const float* __restrict__ delta,
          __nv_bfloat16* __restrict__ dQ,
          float* __restrict__ part, int wide) {
  using C = CfgQ<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1k(smem_raw);
  BarsQ<DP>* bars = reinterpret_cast<BarsQ<DP>*>(smem + C::OFF_BAR);
  const uint32_t sbase = smem_u32(smem);
  const int warp = warp_number(), lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::QST; ++s) mbar_init(&bars->qfull[s], 1), mbar_init(&bars->qempty[s], 1);
    for (int s = 0; s < C::KST; ++s) mbar_init(&bars->kfull[s], 1), mbar_init(&bars->kempty[s], 1);
    for (int s = 0; s < C::VST; ++s) mbar_init(&bars->vfull[s], 1), mbar_init(&bars->vempty[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->sfull[s], 1);
      mbar_init(&bars->dsready[s], MATH_WARPS);
    }
    mbar_init(&bars->dpfull, 1);
    mbar_init(&bars->dpfree, MATH_WARPS);
    mbar_init(&bars->dqfull, 1);
    mbar_init(&bars->dqfree, 4);
    mbar_init(&bars->final_[0], 1);
    mbar_init(&bars->final_[1], 1);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == CTRL + 1) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == CTRL && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmG);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
  pdl_trigger();
  pdl_wait();  // D_i, the gathered keys and their counts

  if (warp >= CTRL) {
    regs_dec<REGS_CTRL>();
    if (warp == CTRL && lane == 0) {
      // ---------------------------------------------------------- TMA producer
      uint32_t qi = 0, ki = 0;
      bool ok = true;
      auto load_q = [&](const CUtensorMap* m, const WorkQ& w) {
        const uint32_t s = qi % C::QST;
        if (!mbar_wait_near(&bars->qempty[s], ((qi / C::QST) & 1) ^ 1, abort_flag)) return false;
        load_tile<DP>(smem + C::OFF_Q + s * C::TILE, m, w.qt * BM, w.h, w.b, &bars->qfull[s]);
        ++qi;
        return true;
      };
      for (WorkQ w = before_first_q(); ok && (w = next_q(a, w)).i < a.total;) {
        const int32_t kh = w.h / a.group;
        for (int j = 0; ok && j < w.nk; ++j, ++ki) {
          const int32_t n = (w.k0 + j) * BN;
          if (j == 0 && !(ok = load_q(&tmQ, w))) break;
          const uint32_t sk = ki % C::KST, sv = ki % C::VST;
          if (!(ok = mbar_wait_near(&bars->kempty[sk], ((ki / C::KST) & 1) ^ 1, abort_flag))) break;
          load_tile<DP>(smem + C::OFF_K + sk * C::TILE, &tmK, n, kh, w.b, &bars->kfull[sk]);
          if (j == 0) ok = load_q(&tmG, w);
          if (ok) ok = mbar_wait_near(&bars->vempty[sv], ((ki / C::VST) & 1) ^ 1, abort_flag);
          if (!ok) {
            mbar_wait_drain(&bars->kfull[sk], (ki / C::KST) & 1);
            break;
          }
          if (!lose(LOSE_DQ_V)) load_tile<DP>(smem + C::OFF_V + sv * C::TILE, &tmV, n, kh, w.b, &bars->vfull[sv]);
        }
      }
      // Every copy lands before the CTA's shared memory goes away, whoever gives up, now or later.
      drain(bars->qfull, C::QST, qi);
      drain(bars->kfull, C::KST, ki);
      drain(bars->vfull, C::VST, ki);
    } else if (warp == CTRL + 1) {
      // ---------------------------------------------------------- MMA issuer of S and dQ
      // (the issuers' warps stay converged; one's waits hide behind the other's products)
      uint32_t i = 0, items = 0;  // steps (key tiles) and items done
      bool ok = true;
      auto issue_s = [&](const WorkQ& w, int j, uint32_t step, uint32_t item) {
        const uint32_t qs = (2 * item) % C::QST, ks = step % C::KST;
        const uint32_t id = xt::idesc_n(BM, static_cast<uint32_t>((keys_of(w, j) + 15) & ~15));
        const uint64_t qd = tile::desc_k(sbase + C::OFF_Q + qs * C::TILE, 0);
        const uint64_t kd = tile::desc_k(sbase + C::OFF_K + ks * C::TILE, 0);
        ok = warp_wait_near(&bars->kfull[ks], (step / C::KST) & 1, abort_flag);
        if (j == 0) ok = ok && warp_wait_near(&bars->qfull[qs], ((2 * item) / C::QST) & 1, abort_flag);
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          tile::mma_kk<DP>(tmem + Q_S + 128u * (step & 1), qd, kd, id);
          mma_commit(&bars->sfull[step & 1]);
          if (j == w.nk - 1) mma_commit(&bars->qempty[qs]);
        }
        __syncwarp();
      };
      WorkQ w, nx = before_first_q();
      for (int first = 1; ok && nx.i < a.total; first = 0) {
        w = nx;
        nx = next_q(a, w);
        // Step -1 of the first turn issues the very first S; every other step the next one's.
        for (int j = -first; ok && j < w.nk; ++j) {
          const bool last = j + 1 >= w.nk;
          const WorkQ& v = last ? nx : w;
          if (v.i < a.total) issue_s(v, last ? 0 : j + 1, i + (1 - first), items + (last && !first ? 1 : 0));
          if (first) break;
          // dQ += ds K
          const int ksteps = (keys_of(w, j) + 15) >> 4;
          const uint32_t ks = i % C::KST;
          const uint64_t kd = tile::desc_mn(sbase + C::OFF_K + ks * C::TILE, 0);
          const uint32_t ds = tmem + Q_S + 128u * (i & 1);
          if (j == 0) ok = ok && warp_wait_near(&bars->dqfree, (items & 1) ^ 1, abort_flag);
          ok = ok && warp_wait_near(&bars->dsready[i & 1], (i >> 1) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll 1
            for (int kk = 0; kk < ksteps; ++kk)
              mma_bf16_ts(tmem + Q_DQ, ds + 8u * (kk & 1) + 32u * (kk >> 1), kd + tile::step_mn(kk),
                          idesc_bf16_f32(BM, DP, false, true), j > 0 || kk > 0);
            mma_commit(&bars->kempty[ks]);
            if (last) mma_commit(&bars->dqfull);
          }
          __syncwarp();
          ++i;
        }
        if (!first) ++items;
      }
      if (elect_one()) mma_commit(&bars->final_[0]);
      __syncwarp();
      mbar_wait_drain(&bars->final_[0], 0);
      __syncwarp();
    } else if (warp == CTRL + 2) {
      // ---------------------------------------------------------- MMA issuer of dP
      uint32_t i = 0, item = 0;
      bool ok = true;
      for (WorkQ w = before_first_q(); ok && (w = next_q(a, w)).i < a.total; ++item) {
        const uint32_t gs = (2 * item + 1) % C::QST;
        const uint64_t gd = tile::desc_k(sbase + C::OFF_Q + gs * C::TILE, 0);
        for (int j = 0; j < w.nk; ++j, ++i) {
          const uint32_t vs = i % C::VST;
          const uint32_t id = xt::idesc_n(BM, static_cast<uint32_t>((keys_of(w, j) + 15) & ~15));
          const uint64_t vd = tile::desc_k(sbase + C::OFF_V + vs * C::TILE, 0);
          if (j == 0) ok = warp_wait_near(&bars->qfull[gs], ((2 * item + 1) / C::QST) & 1, abort_flag);
          ok = ok && warp_wait_near(&bars->vfull[vs], (i / C::VST) & 1, abort_flag);
          // the math warps have read the last dP
          ok = ok && warp_wait_near(&bars->dpfree, (i & 1) ^ 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            tile::mma_kk<DP>(tmem + Q_DP, gd, vd, id);
            mma_commit(&bars->dpfull);
            mma_commit(&bars->vempty[vs]);
            if (j == w.nk - 1) mma_commit(&bars->qempty[gs]);
          }
          __syncwarp();
        }
      }
      if (elect_one()) mma_commit(&bars->final_[1]);
      __syncwarp();
      mbar_wait_drain(&bars->final_[1], 0);
      __syncwarp();
    }
  } else if (warp < MATH_WARPS) {
    // ------------------------------------------------------------ math: p, ds of a quarter of a row
    regs_inc<REGS_MATH>();
    const int cq = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t t_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 32u * cq;
    uint32_t i = 0;
    bool ok = true;
    // An item's lse and D are read while the item before is worked on.
    WorkQ nx = before_first_q();
    // (Only loaded there: a product of what is on its way would wait for it.)
    float lse_next = 0.f, delta_next = 0.f;
    while (ok && nx.i < a.total) {
      const WorkQ w = nx;
      const float nl = -lse_next * LOG2E, nd = -delta_next;
      nx = next_q(a, w);
      if (nx.i < a.total) {
        const int64_t n = int64_t(nx.qt) * BM + row, r = (int64_t(nx.b) * a.H + nx.h) * a.Nq + n;
        lse_next = delta_next = 0.f;
        if (n < a.Nq) {
          lse_next = lse[r];
          delta_next = delta[r];
        }
      }
      const uint64_t c2 = pk(a.c, a.c), nl2 = pk(nl, nl), nd2 = pk(nd, nd);
      for (int j = 0; j < w.nk; ++j, ++i) {
        const int nv = keys_of(w, j) - 32 * cq;  // keys of this quarter
        const uint32_t ts = t_row + Q_S + 128u * (i & 1);
        if (!(ok = warp_wait_near(&bars->sfull[i & 1], (i >> 1) & 1, abort_flag))) break;
        tc_fence_after();
        uint32_t s[32];
        if (nv > 0) {
          tmem_ld_x32(ts, s);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = upk(fma2(pk(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, nl2));
            s[e] = __float_as_uint(exp2_approx(x.x));
            s[e + 1] = __float_as_uint(exp2_approx(x.y));
          }
          if (nv < 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= nv) s[e] = 0;
          }
        }
        if (!(ok = warp_wait_near(&bars->dpfull, i & 1, abort_flag))) break;
        tc_fence_after();
        auto free_dp = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->dpfree);
        };
        if (nv > 0) {
          uint32_t d[16], g[16];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            tmem_ld_x16(t_row + Q_DP + 16 * q, g);
            tmem_ld_wait();
            if (q == 1) free_dp();
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const uint64_t x = add2(pk(__uint_as_float(g[e]), __uint_as_float(g[e + 1])), nd2);
              const float2 y = upk(mul2(x, pk(__uint_as_float(s[16 * q + e]), __uint_as_float(s[16 * q + e + 1]))));
              d[8 * q + e / 2] = pack_bf16(y.x, y.y);
            }
          }
          tmem_st_x16(ts, d);
        } else {
          free_dp();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->dsready[i & 1]);
      }
    }
  } else {
    // ------------------------------------------------------------ dQ to memory
    regs_dec<REGS_AUX>();
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t t_dq = tmem + Q_DQ + (static_cast<uint32_t>(quarter * 32) << 16);
    uint32_t done = 0;  // items with keys whose dQ is stored
#pragma unroll 1
    for (int64_t x = blockIdx.x; x < a.total; x += gridDim.x) {
      const WorkQ w = get_q(a, x);
      const int64_t n = int64_t(w.qt) * BM + row;
      const int64_t r = (int64_t(w.b) * a.H + w.h) * a.Nq + n;
      __nv_bfloat16* o = dQ + w.b * a.dq.b + w.h * a.dq.h + n * a.dq.n;
      float* po = part + (int64_t(w.split) * a.rows + r) * D;
      const bool in = n < a.Nq;
      if (w.nk > 0) {
        if (!warp_wait_near(&bars->dqfull, done & 1, abort_flag)) break;
        ++done;
        tc_fence_after();
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32] = {};
        if (w.nk > 0) {
          tmem_ld_x32(t_dq + 32 * c, v);
          tmem_ld_wait();
        }
        if (in) store_row32(o + 32 * c, po + 32 * c, v, a.scale, a.splits > 1, wide != 0);
      }
      if (w.nk > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->dqfree);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == CTRL + 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------------------------ dK, dV
template <int DP>
struct CfgK {
  static constexpr uint32_t TILE = (DP / 64) * HALF;
  static constexpr int QST = DP == 128 ? 3 : 4;   // Q tiles: one is held until dK has used it
  static constexpr int GST = DP == 128 ? 2 : 4;   // dO tiles, and the queries' lse and D
  static constexpr uint32_t OFF_K = 0;
  static constexpr uint32_t OFF_V = TILE;
  static constexpr uint32_t OFF_Q = 2 * TILE;
  static constexpr uint32_t OFF_G = OFF_Q + QST * TILE;
  static constexpr uint32_t OFF_L = OFF_G + GST * TILE;   // [GST][2][128]: -lse log2(e), -D
  static constexpr uint32_t OFF_BAR = OFF_L + GST * 2 * BM * 4;
  static constexpr uint32_t SMEM = OFF_BAR + 384;  // (the block's shared memory starts on a 1 KB boundary)
};
static_assert(CfgK<128>::SMEM <= 232448 && CfgK<64>::SMEM <= 232448, "shared memory budget");

template <int DP>
struct BarsK {
  uint64_t qfull[CfgK<DP>::QST], qempty[CfgK<DP>::QST];
  uint64_t gfull[CfgK<DP>::GST], gempty[CfgK<DP>::GST];
  uint64_t lfull[CfgK<DP>::GST], lempty[CfgK<DP>::GST];
  uint64_t kfull, kempty, vfull, vempty;
  // S^T of even and odd steps: a wait tells a phase from the one before it only, and the S^T issuer may
  // be a step ahead of the other one, which waits for it too (S^T(i + 2) wants p(i + 1), which wants
  // nothing of dP).  It cannot be three steps ahead: p(i + 2) wants dP(i + 1), which comes after that wait.
  uint64_t sfull[2];
  uint64_t pready, dpfull, dsready, accfull, accfree, final_[2];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(BarsK<64>) <= 384, "barrier block too large");

constexpr uint32_t K_S = 0, K_DP = 128, K_DV = 256, K_DK = 384;

struct WorkK {
  int64_t i;
  int32_t b, h, kt, split;   // h: key head
  int32_t t0, nq, keys;      // first query tile of the group, query tiles; 0: no keys in the tile
};
__device__ __forceinline__ WorkK get_k(const Args& a, int64_t i) {
  WorkK w;
  w.i = i;
  uint32_t r = static_cast<uint32_t>(i);
  const uint32_t q = fdiv(r, a.fd_tiles);
  w.kt = static_cast<int32_t>(r - q * a.tiles);
  r = fdiv(q, a.fd_splits);
  w.split = static_cast<int32_t>(q - r * a.splits);
  w.b = static_cast<int32_t>(fdiv(r, a.fd_heads));
  w.h = static_cast<int32_t>(r - w.b * static_cast<uint32_t>(a.Hkv));
  w.keys = a.count ? __ldg(a.count + w.b) : static_cast<int32_t>(a.Nk);
  w.t0 = w.split * a.per;
  const int32_t tiles = a.q_tiles * a.group - w.t0;
  w.nq = tiles < a.per ? tiles : a.per;
  if (w.nq < 0 || int64_t(w.kt) * BN >= w.keys) w.nq = 0;
  return w;
}
// The item before this CTA's first, and the next one with work.
__device__ __forceinline__ WorkK before_first_k() {
  WorkK w;
  w.i = int64_t(blockIdx.x) - gridDim.x;
  w.nq = 0;
  return w;
}
__device__ __forceinline__ WorkK next_k(const Args& a, WorkK w) {
#pragma unroll 1
  do {
    w.i += gridDim.x;
    if (w.i >= a.total) break;
    w = get_k(a, w.i);
  } while (w.nq == 0);
  return w;
}

template <int DP, int D>
__global__ void __launch_bounds__(THREADS, 1)
dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
           const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
           const __grid_constant__ Args a, const float* __restrict__ lse, const float* __restrict__ delta,
           float* __restrict__ part_k, float* __restrict__ part_v) {
  using C = CfgK<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // (never: no static shared memory stands before it)
    if (threadIdx.x == 0) atomicOr(&g_la_error, ERR_SMEM_ALIGN);
    return;
  }
  BarsK<DP>* bars = reinterpret_cast<BarsK<DP>*>(smem + C::OFF_BAR);
  const uint32_t sbase = smem_u32(smem);
  float* l_sm = reinterpret_cast<float*>(smem + C::OFF_L);
  const int warp = warp_number(), lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::QST; ++s) {
      mbar_init(&bars->qfull[s], 1);
      mbar_init(&bars->qempty[s], 2);  // both issuers
    }
    for (int s = 0; s < C::GST; ++s) {
      mbar_init(&bars->gfull[s], 1);
      mbar_init(&bars->gempty[s], 2);
      mbar_init(&bars->lfull[s], 4);
      mbar_init(&bars->lempty[s], MATH_WARPS);
    }
    mbar_init(&bars->kfull, 1);
    mbar_init(&bars->kempty, 1);
    mbar_init(&bars->vfull, 1);
    mbar_init(&bars->vempty, 1);
    mbar_init(&bars->sfull[0], 1);
    mbar_init(&bars->sfull[1], 1);
    mbar_init(&bars->pready, MATH_WARPS);
    mbar_init(&bars->dpfull, 1);
    mbar_init(&bars->dsready, MATH_WARPS);
    mbar_init(&bars->accfull, 2);
    mbar_init(&bars->accfree, MATH_WARPS);
    mbar_init(&bars->final_[0], 1);
    mbar_init(&bars->final_[1], 1);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == CTRL + 1) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == CTRL && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmG);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
  pdl_trigger();
  pdl_wait();  // D_i, the gathered keys and their counts (every kernel of the chain has waited for the one before)

  if (warp >= CTRL) {
    regs_dec<REGS_CTRL>();
    if (warp == CTRL && lane == 0) {
      // ---------------------------------------------------------- TMA producer
      uint32_t qi = 0, items = 0;
      uint32_t k_out = 0, v_out = 0;
      bool ok = true;
      for (WorkK w = before_first_k(); ok && (w = next_k(a, w)).i < a.total; ++items) {
        if (!(ok = mbar_wait_near(&bars->kempty, (items & 1) ^ 1, abort_flag))) break;
        load_tile<DP>(smem + C::OFF_K, &tmK, w.kt * BN, w.h, w.b, &bars->kfull);
        ++k_out;
        for (int j = 0; ok && j < w.nq; ++j, ++qi) {
          const int32_t it = w.t0 + j, hq = it / a.q_tiles;
          const int32_t h = w.h * a.group + hq, n = (it - hq * a.q_tiles) * BM;
          const uint32_t s = qi % C::QST, sg = qi % C::GST;
          if (!(ok = mbar_wait_near(&bars->qempty[s], ((qi / C::QST) & 1) ^ 1, abort_flag))) break;
          load_tile<DP>(smem + C::OFF_Q + s * C::TILE, &tmQ, n, h, w.b, &bars->qfull[s]);
          if (j == 0) {
            ok = mbar_wait_near(&bars->vempty, (items & 1) ^ 1, abort_flag);
            if (ok) {
              load_tile<DP>(smem + C::OFF_V, &tmV, w.kt * BN, w.h, w.b, &bars->vfull);
              ++v_out;
            }
          }
          if (ok) ok = mbar_wait_near(&bars->gempty[sg], ((qi / C::GST) & 1) ^ 1, abort_flag);
          if (!ok) {
            mbar_wait_drain(&bars->qfull[s], (qi / C::QST) & 1);
            break;
          }
          hold(HOLD_DO_LOAD);
          if (!lose(LOSE_DKV_DO)) load_tile<DP>(smem + C::OFF_G + sg * C::TILE, &tmG, n, h, w.b, &bars->gfull[sg]);
        }
        if (!ok) break;
      }
      // (as in dq_kernel)
      drain(bars->qfull, C::QST, qi);
      drain(bars->gfull, C::GST, qi);
      drain(&bars->kfull, 1, k_out);
      drain(&bars->vfull, 1, v_out);
    } else if (warp == CTRL + 1 || warp == CTRL + 2) {
      // ---------------------------------------------------------- MMA issuers (converged warps)
      // The first: S^T and dV, the second: dP^T and dK.  Each walks the same steps: the product of this
      // step's p (ds) first, then the scores (dP) of the next step, which overwrite it.
      const bool sv = warp == CTRL + 1;
      uint32_t i = 0, items = 0;
      bool ok = true;
      const uint32_t id_s = idesc_bf16_f32(BM, BN, false, false), id_d = idesc_bf16_f32(BM, DP, false, true);
      const uint32_t t_in = tmem + (sv ? K_S : K_DP), t_acc = tmem + (sv ? K_DV : K_DK);
      const uint32_t fixed = sbase + (sv ? C::OFF_K : C::OFF_V);          // the item's K (V) tile
      const uint32_t in = sbase + (sv ? C::OFF_Q : C::OFF_G);             // ... times Q (dO) tiles
      const uint32_t out = sbase + (sv ? C::OFF_G : C::OFF_Q);            // p dO (ds Q)
      uint64_t* in_full = sv ? bars->qfull : bars->gfull;
      uint64_t* out_full = sv ? bars->gfull : bars->qfull;
      uint64_t* in_empty = sv ? bars->qempty : bars->gempty;
      uint64_t* out_empty = sv ? bars->gempty : bars->qempty;
      uint64_t* fixed_full = sv ? &bars->kfull : &bars->vfull;
      uint64_t* fixed_empty = sv ? &bars->kempty : &bars->vempty;
      uint64_t* ready = sv ? &bars->pready : &bars->dsready;
      const uint32_t in_st = sv ? C::QST : C::GST, out_st = sv ? C::GST : C::QST;
      const uint64_t fd = tile::desc_k(fixed, 0);
      auto issue_in = [&](bool last, uint32_t s, uint32_t step) {
        tile::mma_kk<DP>(t_in, fd, tile::desc_k(in + s * C::TILE, 0), id_s);
        mma_commit(sv ? &bars->sfull[step & 1] : &bars->dpfull);
        mma_commit(&in_empty[s]);
        if (last) mma_commit(fixed_empty);
      };
      WorkK w, nx = before_first_k();
      for (int first = 1; ok && nx.i < a.total; first = 0) {
        w = nx;
        nx = next_k(a, w);
        if (first) {  // the first scores; the others follow the product before them
          if (nx.i >= a.total) break;
          ok = warp_wait_near(fixed_full, 0, abort_flag) && warp_wait_near(&in_full[0], 0, abort_flag);
          tc_fence_after();
          if (ok && elect_one()) issue_in(nx.nq == 1, 0, 0);
          __syncwarp();
          continue;
        }
        for (int j = 0; ok && j < w.nq; ++j, ++i) {
          const bool last = j + 1 == w.nq, more = !last || nx.i < a.total;
          const bool last2 = last ? nx.nq == 1 : j + 2 == w.nq;
          const uint32_t s = i % out_st, s2 = (i + 1) % in_st;
          const uint64_t od = tile::desc_mn(out + s * C::TILE, 0);
          if (more) {
            if (last) ok = warp_wait_near(fixed_full, (items + 1) & 1, abort_flag);
            ok = ok && warp_wait_near(&in_full[s2], ((i + 1) / in_st) & 1, abort_flag);
          }
          if (j == 0) ok = ok && warp_wait_near(&bars->accfree, (items & 1) ^ 1, abort_flag);
          // This step's dO (Q) tile: p is ready from S^T and the exponentials alone, and loads land in any
          // order, so neither it nor the next Q tile says that dO is there.
          ok = ok && warp_wait_near(&out_full[s], (i / out_st) & 1, abort_flag);
          ok = ok && warp_wait_near(ready, i & 1, abort_flag);
          // The next p waits for the next S^T: dV and S^T have the tensor cores to themselves first.
          if (!sv) hold(HOLD_DP_ISSUER);
          if (!sv && more) ok = ok && warp_wait_near(&bars->sfull[(i + 1) & 1], ((i + 1) >> 1) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < BM / 16; ++kk)
              mma_bf16_ts(t_acc, t_in + 8u * (kk & 1) + 32u * (kk >> 1), od + tile::step_mn(kk), id_d, j > 0 || kk > 0);
            mma_commit(&out_empty[s]);
            if (last) mma_commit(&bars->accfull);
            if (more) issue_in(last2, s2, i + 1);
          }
          __syncwarp();
        }
        ++items;
      }
      if (elect_one()) mma_commit(&bars->final_[sv ? 0 : 1]);
      __syncwarp();
      mbar_wait_drain(&bars->final_[sv ? 0 : 1], 0);
      __syncwarp();
    }
  } else if (warp < MATH_WARPS) {
    // ------------------------------------------------------------ math: p, ds of a quarter of a key's row
    regs_inc<REGS_MATH>();
    const int cq = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t t_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t ts = t_row + K_S + 32u * cq, tp = t_row + K_DP + 32u * cq;
    const uint64_t c2 = pk(a.c, a.c);
    uint32_t i = 0, item = 0;
    bool ok = true;
    for (WorkK w = before_first_k(); ok && (w = next_k(a, w)).i < a.total; ++item) {
      for (int j = 0; j < w.nq; ++j, ++i) {
        const uint32_t s_l = i % C::GST;
        const uint32_t la_ = sbase + C::OFF_L + (s_l * 2 * BM + 32 * cq) * 4, ld_ = la_ + BM * 4;
        if (!(ok = warp_wait_near(&bars->lfull[s_l], (i / C::GST) & 1, abort_flag))) break;
        if (!(ok = warp_wait_near(&bars->sfull[i & 1], (i >> 1) & 1, abort_flag))) break;
        tc_fence_after();
        uint32_t s[32], d[16];
        tmem_ld_x32(ts, s);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 nl = lds128f(la_ + e * 4);
          const float2 x = upk(fma2(pk(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, pk(nl.x, nl.y)));
          const float2 y = upk(fma2(pk(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), c2, pk(nl.z, nl.w)));
          const float p0 = exp2_approx(x.x), p1 = exp2_approx(x.y), p2 = exp2_approx(y.x), p3 = exp2_approx(y.y);
          s[e] = __float_as_uint(p0);
          s[e + 1] = __float_as_uint(p1);
          s[e + 2] = __float_as_uint(p2);
          s[e + 3] = __float_as_uint(p3);
          d[e / 2] = pack_bf16(p0, p1);
          d[e / 2 + 1] = pack_bf16(p2, p3);
        }
        tmem_st_x16(ts, d);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->pready);
        if (!(ok = warp_wait_near(&bars->dpfull, i & 1, abort_flag))) break;
        tc_fence_after();
        uint32_t g[16];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          tmem_ld_x16(tp + 16 * q, g);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 nd = lds128f(ld_ + (16 * q + e) * 4);
            const int k = 16 * q + e;
            const float2 x = upk(mul2(add2(pk(__uint_as_float(g[e]), __uint_as_float(g[e + 1])), pk(nd.x, nd.y)),
                                      pk(__uint_as_float(s[k]), __uint_as_float(s[k + 1]))));
            const float2 y = upk(mul2(add2(pk(__uint_as_float(g[e + 2]), __uint_as_float(g[e + 3])), pk(nd.z, nd.w)),
                                      pk(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3]))));
            d[k / 2] = pack_bf16(x.x, x.y);
            d[k / 2 + 1] = pack_bf16(y.x, y.y);
          }
        }
        tmem_st_x16(tp, d);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars->dsready);
          mbar_arrive(&bars->lempty[s_l]);
        }
      }
      if (!ok) break;
      // the item's sums, a key per thread: warps 0-7 store dV, 8-15 dK, half of the channels each
      if (!(ok = warp_wait_near(&bars->accfull, item & 1, abort_flag))) break;
      tc_fence_after();
      const int64_t n = int64_t(w.kt) * BN + row;
      const bool is_v = cq < 2;
      const float f = is_v ? 1.f : a.scale;
      float* out = (is_v ? part_v : part_k) + (int64_t(w.split) * a.keys + (int64_t(w.b) * a.Hkv + w.h) * a.Nk + n) * D;
      const uint32_t ta = t_row + (is_v ? K_DV : K_DK);
#pragma unroll 1
      for (int c = cq & 1; c < D / 32; c += 2) {
        uint32_t v[32];
        tmem_ld_x32(ta + 32 * c, v);
        tmem_ld_wait();
        if (n < w.keys) store_row32(nullptr, out + 32 * c, v, f, true, true);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->accfree);
    }
  } else {
    // ------------------------------------------------------------ -lse log2(e) and -D of the queries
    regs_dec<REGS_AUX>();
    const int q = (warp & 3) * 32 + lane;
    uint32_t i = 0;
    bool ok = true;
    for (WorkK w = before_first_k(); ok && (w = next_k(a, w)).i < a.total;) {
      for (int j = 0; j < w.nq; ++j, ++i) {
        const uint32_t s = i % C::GST;
        const int32_t it = w.t0 + j, hq = it / a.q_tiles;
        const int64_t n = int64_t(it - hq * a.q_tiles) * BM + q;
        const int64_t r = (int64_t(w.b) * a.H + w.h * a.group + hq) * a.Nq + n;
        // queries past the end: p = 2^-inf = 0
        const float nl = n < a.Nq ? -lse[r] * LOG2E : xs::NEG_INF, nd = n < a.Nq ? -delta[r] : 0.f;
        if (!(ok = warp_wait_near(&bars->lempty[s], ((i / C::GST) & 1) ^ 1, abort_flag))) break;
        l_sm[s * 2 * BM + q] = nl;
        l_sm[s * 2 * BM + BM + q] = nd;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->lfull[s]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == CTRL + 1) tmem_dealloc(tmem, 512);
}

}  // namespace xb
}  // namespace la
