// cross_tc.cuh -- cross attention forward on the 5th-generation tensor cores (bf16).
//
//   s_ij = scale q_i.k_j,  o_i = sum_j exp(s_ij - lse_i) v_j
//
// A CTA works on two tiles of 128 queries at a time and walks the keys in tiles of 128.  Per query
// tile and key tile: S = Q K^T (accumulator in tensor memory), the softmax warps read a row each,
// keep its running maximum and sum in registers and write P = 2^(S c - m) back to tensor memory as
// bf16 (rounded once; the sum takes the unrounded values), and O += P V with P as the operand in
// tensor memory.  The two query tiles alternate, so that the tensor cores work on one while the
// exponentials of the other are computed: their warps on a scheduler take turns at those.  With c = scale log2(e) and a reference maximum m that is
// only raised when a row's maximum has grown by more than 2^8 (then O and the sum are rescaled),
// the accumulator is hardly ever touched between the first and the last key tile.
// The last key tile is cut to a multiple of 16 keys in both products and to a multiple of 32 in the
// softmax.
//
// 32 heads at 1965 MHz: 75600 queries and 300 keys 442 us (840 TFLOP/s, 2.8 TB/s), 8192 x 8192 986 us (1115
// TFLOP/s of the 1684 that a large matrix product reaches).  At 8192 x 8192 a tile of 128 x 128 scores takes
// 2190 cycles, with half the channels 2060: its products 1450 (725) at that rate, its exponentials 1024.  So
// the softmax warps bound it: a turn has one warp a scheduler, which scales, converts, loads and stores
// too, and the exponentials' unit runs at half its rate.  Short keys add the epilogue of every 3 key tiles.
//
// Warps (one CTA per SM, persistent; work item = pair of query tiles of a head, or a part of its
// keys where there are too few items):
//   0-3, 4-7   softmax of query tile 0 / 1 (thread = row)
//   8-11       epilogue: O / sum to global memory, a row per thread in 32-byte stores
//   12         TMA producer
//   13, 14     MMA issuers of query tile 0 / 1 (15 completes the warpgroup)
// Tensor memory: S (and P) of the two tiles in columns [0, 256), O in [256, 512).
// Every wait is bounded (mbar_wait_near), and no barrier completes two phases ahead of anyone who waits
// for it: a slot is filled again after its issuers (K and V: both) have given it back, S after all of a
// tile's softmax warps have arrived, P and O after a product that the waiting issuer issues behind its
// wait, a turn after the other tile's, inv_l after the epilogue has read the last one.
#pragma once
#include "common.cuh"
#include "cross_simt.cuh"
#include "sm100.cuh"
#include "tile_ops.cuh"

namespace la {
namespace xt {

constexpr int BM = 128, BN = 128;
constexpr int THREADS = 512;
constexpr int QST = 3;  // query tiles in shared memory: the two at work and the next one
constexpr uint32_t HALF = 128 * 128;  // bytes of 128 rows of 64 channels
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float RESCALE = 8.f;  // P stays below 2^8, its sum below Nk 2^8: far inside fp32 and bf16

template <int DP>
struct Cfg {
  static constexpr uint32_t TILE = (DP / 64) * HALF;
  static constexpr int KVST = DP == 128 ? 4 : 8;  // key and value tiles in flight
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_KV = QST * TILE;
  static constexpr uint32_t OFF_L = OFF_KV + KVST * TILE;
  static constexpr uint32_t OFF_BAR = OFF_L + 2 * BM * 4;
  static constexpr uint32_t SMEM = OFF_BAR + 512 + 1024;
};
static_assert(Cfg<128>::SMEM <= 232448 && Cfg<64>::SMEM <= 232448, "shared memory budget");

constexpr uint32_t S_COL = 0, O_COL = 256;  // + 128 t
// Registers: 128 a thread at launch (the host checks that), handed on to the softmax warps.
constexpr uint32_t REGS_LAUNCH = 128, REGS_SOFTMAX = 152, REGS_EPI = 128, REGS_CTRL = 80;
static_assert(256 * REGS_SOFTMAX + 128 * REGS_EPI + 128 * REGS_CTRL <= THREADS * REGS_LAUNCH, "register split");

template <int DP>
struct Bars {
  uint64_t qfull[QST], qempty[QST];
  uint64_t kvfull[Cfg<DP>::KVST], kvempty[Cfg<DP>::KVST];
  uint64_t order[2][4];
  uint64_t sfull[2], pready[2], pvdone[2], ofull[2], ofree[2], lready[2];
  uint64_t final_[2];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Bars<64>) <= 512, "barrier block too large");

struct Args {
  int64_t B, H, Nq, Nk, rows;
  int64_t total;          // work items: B * H * splits * pairs
  int32_t pairs;          // pairs of query tiles per head
  int32_t group;          // query heads per key head
  int32_t splits, per;    // parts of the keys, key tiles per part
  FastDiv fd_pairs, fd_splits, fd_H;
  float c;                // scale * log2(e)
  const int32_t* count;   // keys per batch row (gathered), or null: Nk
  xs::Str o;
};

// Instruction descriptor of a product with M rows and n columns (a multiple of 16), both operands
// K-major.
__device__ __forceinline__ uint32_t idesc_n(uint32_t M, uint32_t n) {
  return idesc_bf16_f32(M, 0, false, false) | ((n >> 3) << 17);
}

struct Work {
  int64_t i;
  int32_t b, h, pair, split;
  int32_t k0, nk;   // first key tile, key tiles (0: nothing attended in this part)
  int32_t keys;     // attended keys of the batch row
  int32_t nt;       // query tiles with rows
};

__device__ __forceinline__ Work get_work(const Args& a, int64_t i) {
  Work w;
  w.i = i;
  uint32_t r = static_cast<uint32_t>(i);
  const uint32_t q = fdiv(r, a.fd_pairs);
  w.pair = static_cast<int32_t>(r - q * a.pairs);
  r = fdiv(q, a.fd_splits);
  w.split = static_cast<int32_t>(q - r * a.splits);
  w.b = static_cast<int32_t>(fdiv(r, a.fd_H));
  w.h = static_cast<int32_t>(r - w.b * static_cast<uint32_t>(a.H));
  w.keys = a.count ? __ldg(a.count + w.b) : static_cast<int32_t>(a.Nk);
  const int32_t tiles = (w.keys + BN - 1) / BN;
  w.k0 = w.split * a.per;
  w.nk = tiles - w.k0 < a.per ? tiles - w.k0 : a.per;
  if (w.nk < 0) w.nk = 0;
  w.nt = int64_t(w.pair) * 2 * BM + BM < a.Nq ? 2 : 1;
  return w;
}
// The item before this CTA's first, and the next one that has keys (i >= total: none).  (The roles
// call next_work in one place each: its code is inlined at every call.)
__device__ __forceinline__ Work before_first() {
  Work w;
  w.i = int64_t(blockIdx.x) - gridDim.x;
  w.nk = w.nt = 0;
  return w;
}
__device__ __forceinline__ Work next_work(const Args& a, Work w) {
#pragma unroll 1
  do {
    w.i += gridDim.x;
    if (w.i >= a.total) break;
    w = get_work(a, w.i);
  } while (w.nk == 0);
  return w;
}
// Attended keys in key tile j of an item.
__device__ __forceinline__ int tile_keys(const Work& w, int j) {
  const int left = w.keys - (w.k0 + j) * BN;
  return left < BN ? left : BN;
}

// A position in a ring of n stages and the parity of its round.
struct Ring {
  uint32_t s, ph;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++s == n) {
      s = 0;
      ph ^= 1;
    }
  }
};

template <uint32_t R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <uint32_t R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// The running maximum over up to 32 scores (n of them attended).
__device__ __forceinline__ void row_max(uint32_t (&s)[32], int n, float (&mx)[4]) {
  if (n < 32) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i >= n) s[i] = __float_as_uint(xs::NEG_INF);
  }
#pragma unroll
  for (int i = 0; i < 32; i += 2)
    mx[(i / 2) & 3] = max3(mx[(i / 2) & 3], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
}
// p = 2^(s c - m) of 32 scores (0 past the n-th), as bf16 to tensor memory; adds to the sums.
__device__ __forceinline__ void row_exp(uint32_t (&s)[32], int n, uint64_t c2, uint64_t m2, uint64_t (&sum)[2], uint32_t to) {
  if (n < 32) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i >= n) s[i] = __float_as_uint(xs::NEG_INF);
  }
  uint32_t p[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint64_t x2 = fma2(pk(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, m2);
    const float2 x = upk(x2), e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
    sum[i & 1] = add2(sum[i & 1], pk(e.x, e.y));
    p[i] = pack_bf16(e.x, e.y);
  }
  tmem_st_x16(to, p);
}

// 32 fp32 channels of a row, times f: as bf16 to o, or (part) as they are to po.
__device__ __forceinline__ void store_row32(__nv_bfloat16* o, float* po, const uint32_t (&v)[32], float f, bool part, bool wide) {
  if (part) {
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
      uint32_t u[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(__uint_as_float(v[e + k]) * f);
      store32(po + e, u, true);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; e += 16) {
      uint32_t u[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        u[k] = pack_bf16(__uint_as_float(v[e + 2 * k]) * f, __uint_as_float(v[e + 2 * k + 1]) * f);
      store32(o + e, u, wide);
    }
  }
}

// DP: channels as the tensor cores see them (64 or 128); D: channels of the tensors (32 runs as 64
// with zeros, which the loads fill in).
template <int DP, int D>
__global__ void __launch_bounds__(THREADS, 1)
forward_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Args a, __nv_bfloat16* __restrict__ O,
               float* __restrict__ lse, float* __restrict__ part_o, float2* __restrict__ part_ml, int wide) {
  using C = Cfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1k(smem_raw);
  Bars<DP>* bars = reinterpret_cast<Bars<DP>*>(smem + C::OFF_BAR);
  const uint32_t sbase = smem_u32(smem);
  float* inv_l = reinterpret_cast<float*>(smem + C::OFF_L);
  const int warp = warp_number(), lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < QST; ++s) {
      mbar_init(&bars->qfull[s], 1);
      mbar_init(&bars->qempty[s], 1);
    }
    for (int s = 0; s < C::KVST; ++s) {
      mbar_init(&bars->kvfull[s], 1);
      mbar_init(&bars->kvempty[s], 2);  // both issuers
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->sfull[t], 1);
      mbar_init(&bars->pready[t], 4);
      for (int q = 0; q < 4; ++q) mbar_init(&bars->order[t][q], 1);
      mbar_init(&bars->pvdone[t], 1);
      mbar_init(&bars->ofull[t], 1);
      mbar_init(&bars->ofree[t], 4);
      mbar_init(&bars->lready[t], 4);
      mbar_init(&bars->final_[t], 1);
    }
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == 12 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
  pdl_trigger();
  pdl_wait();  // the gathered keys and their counts

  if (warp >= 12) {
    regs_dec<REGS_CTRL>();
    if (warp == 12 && lane == 0) {
      // ---------------------------------------------------------- TMA producer
      uint32_t qi = 0, ki = 0;
      bool ok = true;
      auto load_kv = [&](const CUtensorMap* m, const Work& w, int j) {
        const uint32_t s = ki % C::KVST;
        if (!mbar_wait_near(&bars->kvempty[s], ((ki / C::KVST) & 1) ^ 1, abort_flag)) return false;
        uint8_t* dst = smem + C::OFF_KV + s * C::TILE;
        mbar_arrive_expect_tx(&bars->kvfull[s], C::TILE);
        const int32_t n = (w.k0 + j) * BN, h = w.h / a.group;
        ++ki;
        if (m == &tmV && lose(LOSE_FORWARD_V)) return true;
        tma_load_4d(dst, m, 0, n, h, w.b, &bars->kvfull[s]);
        if (DP == 128) tma_load_4d(dst + HALF, m, 64, n, h, w.b, &bars->kvfull[s]);
        return true;
      };
      Work w = before_first();
      while (ok && (w = next_work(a, w)).i < a.total) {
        // Q0, K0, Q1, V0, then K and V of the other key tiles in turn
        const int loads = w.nt + 2 * w.nk;
#pragma unroll 1
        for (int e = 0, t = 0, x = 0; ok && e < loads; ++e) {
          if (t < w.nt && (e == 0 || e == 2)) {
            const uint32_t s = qi % QST;
            if (!(ok = mbar_wait_near(&bars->qempty[s], ((qi / QST) & 1) ^ 1, abort_flag))) break;
            uint8_t* dst = smem + C::OFF_Q + s * C::TILE;
            mbar_arrive_expect_tx(&bars->qfull[s], C::TILE);
            const int32_t n = (w.pair * 2 + t) * BM;
            tma_load_4d(dst, &tmQ, 0, n, w.h, w.b, &bars->qfull[s]);
            if (DP == 128) tma_load_4d(dst + HALF, &tmQ, 64, n, w.h, w.b, &bars->qfull[s]);
            ++qi;
            ++t;
          } else {
            ok = load_kv((x & 1) ? &tmV : &tmK, w, x >> 1);
            ++x;
          }
        }
      }
      // Every copy lands before the CTA's shared memory goes away, whoever gives up, now or later.
      for (uint32_t j = (qi > QST ? qi - QST : 0); j < qi; ++j) mbar_wait_drain(&bars->qfull[j % QST], (j / QST) & 1);
      for (uint32_t j = (ki > C::KVST ? ki - C::KVST : 0); j < ki; ++j)
        mbar_wait_drain(&bars->kvfull[j % C::KVST], (j / C::KVST) & 1);
    } else if (warp == 13 || warp == 14) {
      // ---------------------------------------------------------- MMA issuers, one for each query tile
      // (so that one's waits and bookkeeping hide behind the other's products).  The warp stays
      // converged; what does not depend on P is waited for and computed before P is.
      const int t = warp - 13;
      Ring k = {0, 0}, q = {0, 0};  // K and V tiles (they share a ring), Q tiles
      uint32_t step = 0, item = 0;
      bool ok = true;
      const uint32_t ps = tmem + S_COL + 128u * t, po = tmem + O_COL + 128u * t;
      constexpr uint32_t id_o = idesc_bf16_f32(BM, DP, false, true);
      auto id_s = [&](const Work& w, int j) { return idesc_n(BM, static_cast<uint32_t>((tile_keys(w, j) + 15) & ~15)); };
      auto s_mma = [&](uint64_t qd, uint64_t kd, uint32_t id) {
        tile::mma_kk<DP>(ps, qd, kd, id);
        mma_commit(&bars->sfull[t]);
      };
      // The slot of this issuer's Q tile of an item; the ring moves past all of the item's.
      auto q_slot = [&](const Work& w) {
        Ring mine = q;
        q.next(QST);
        if (w.nt == 2) {
          if (t == 1) mine = q;
          q.next(QST);
        }
        return mine;
      };
      Work w, nx = before_first();
      uint32_t qs = 0;
      for (bool first = true; ok; first = false) {
        w = nx;
        if (w.i >= a.total) break;
        nx = next_work(a, w);
        if (first) {  // the first S; the others follow the product before them
          if (nx.i >= a.total) break;
          ok = warp_wait_near(&bars->kvfull[0], 0, abort_flag);
          const Ring mine = q_slot(nx);
          qs = mine.s;
          if (t < nx.nt) {
            ok = ok && warp_wait_near(&bars->qfull[qs], mine.ph, abort_flag);
            tc_fence_after();
            if (ok && elect_one()) {
              s_mma(tile::desc_k(sbase + C::OFF_Q + qs * C::TILE, 0), tile::desc_k(sbase + C::OFF_KV, 0), id_s(nx, 0));
              if (nx.nk == 1) mma_commit(&bars->qempty[qs]);
              mma_commit(&bars->kvempty[0]);
            }
            __syncwarp();
          } else if (ok && lane == 0) {
            mbar_arrive(&bars->kvempty[0]);
          }
          k.next(C::KVST);
          continue;
        }
        for (int j = 0; ok && j < w.nk; ++j) {
          const bool last = j + 1 == w.nk;
          const bool more = !last || nx.i < a.total;       // a K tile follows
          const bool now = t < w.nt, then = last ? more && t < nx.nt : now;  // this tile takes part
          const Ring v = k;
          k.next(C::KVST);
          const Ring k2 = k;
          if (more) k.next(C::KVST);
          ok = warp_wait_near(&bars->kvfull[v.s], v.ph, abort_flag);
          if (more) ok = ok && warp_wait_near(&bars->kvfull[k2.s], k2.ph, abort_flag);
          if (last && more) {
            const Ring mine = q_slot(nx);
            if (then) {
              qs = mine.s;
              ok = ok && warp_wait_near(&bars->qfull[mine.s], mine.ph, abort_flag);
            }
          }
          const uint64_t vd = tile::desc_mn(sbase + C::OFF_KV + v.s * C::TILE, 0);
          const uint64_t kd = tile::desc_k(sbase + C::OFF_KV + k2.s * C::TILE, 0);
          const uint64_t qd = tile::desc_k(sbase + C::OFF_Q + qs * C::TILE, 0);
          const int ksteps = (tile_keys(w, j) + 15) >> 4;
          const uint32_t ids = last ? id_s(nx, 0) : id_s(w, j + 1);
          const bool q_done = last ? nx.nk == 1 : j + 2 == w.nk;  // the next S is the last one of its Q tile
          if (now) {
            // O_t += P_t V (first of an item: the epilogue has read the last item's O_t)
            if (j == 0) ok = ok && warp_wait_near(&bars->ofree[t], (item & 1) ^ 1, abort_flag);
            ok = ok && warp_wait_near(&bars->pready[t], step & 1, abort_flag);
          }
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (now) {
#pragma unroll 1
              for (int kk = 0; kk < ksteps; ++kk) mma_bf16_ts(po, ps + 8u * kk, vd + tile::step_mn(kk), id_o, j > 0 || kk > 0);
              mma_commit(&bars->pvdone[t]);
            }
            if (then) s_mma(qd, kd, ids);
            if (now) {
              if (last) mma_commit(&bars->ofull[t]);
              mma_commit(&bars->kvempty[v.s]);
            } else {
              mbar_arrive(&bars->kvempty[v.s]);
            }
            if (then) {
              if (q_done) mma_commit(&bars->qempty[qs]);
              mma_commit(&bars->kvempty[k2.s]);
            } else if (more) {
              mbar_arrive(&bars->kvempty[k2.s]);
            }
          }
          __syncwarp();
          if (now) {
            ++step;
            if (last) ++item;
          }
        }
      }
      if (elect_one()) mma_commit(&bars->final_[t]);
      __syncwarp();
      mbar_wait_drain(&bars->final_[t], 0);
      __syncwarp();
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax, one row per thread
    regs_inc<REGS_SOFTMAX>();
    const int t = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + S_COL + 128u * t + lane_bits;
    const uint32_t to = tmem + O_COL + 128u * t + lane_bits;
    uint32_t step = 0, item = 0, turn = 0;
    bool ok = true;
    Work nx = before_first();
    while (ok && nx.i < a.total) {
      const Work w = nx;
      nx = next_work(a, w);
      if (t >= w.nt) continue;  // (also before the first)
      float m = 0.f, l = 0.f;
      for (int j = 0; j < w.nk; ++j, ++step) {
        const int nv = tile_keys(w, j);
        if (!(ok = warp_wait_near(&bars->sfull[t], step & 1, abort_flag))) break;
        tc_fence_after();
        // Two passes over the row in chunks of 32 scores, by small loops: the code stays within the
        // instruction cache, and a row needs 64 registers instead of 128.
        const int nc = (nv + 31) >> 5;
        float mx[4] = {xs::NEG_INF, xs::NEG_INF, xs::NEG_INF, xs::NEG_INF};
        uint32_t s0[32], s1[32];
#pragma unroll 1
        for (int c = 0; c < nc; c += 2) {
          tmem_ld_x32(ts + 32 * c, s0);
          if (c + 1 < nc) tmem_ld_x32(ts + 32 * c + 32, s1);
          tmem_ld_wait();
          row_max(s0, nv - 32 * c, mx);
          if (c + 1 < nc) row_max(s1, nv - 32 * c - 32, mx);
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.c;
        tmem_ld_x32(ts, s0);
        if (j == 0) {
          m = fmaxf(top, xs::LOWEST);  // (scores of -inf only, so far)
        } else if (__any_sync(0xffffffffu, top > m + RESCALE)) {
          // rare: raise the reference maximum of the rows that need it
          const float m2 = top > m + RESCALE ? top : m;
          const float f = exp2_approx(m - m2);
          m = m2;
          l *= f;
          if (!(ok = warp_wait_near(&bars->pvdone[t], (step - 1) & 1, abort_flag))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < DP / 16; ++c) {
            uint32_t o[16];
            tmem_ld_x16(to + 16 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st_x16(to + 16 * c, o);
          }
        }
        const uint64_t c2 = pk(a.c, a.c), m2 = pk(-m, -m);
        uint64_t sum[2] = {0, 0};
        // The two tiles' warps on a scheduler take turns at the exponentials: one tile's run while the
        // other's products do, instead of both at once at half the rate.
        if (w.nt == 2 && !(ok = warp_wait_near(&bars->order[t][quarter], t == 0 ? (turn & 1) ^ 1 : turn & 1, abort_flag))) break;
#pragma unroll 1
        for (int c = 0; c < nc; c += 2) {
          tmem_ld_wait();
          if (c + 1 < nc) tmem_ld_x32(ts + 32 * c + 32, s1);
          row_exp(s0, nv - 32 * c, c2, m2, sum, ts + 16 * c);
          if (c + 1 < nc) {
            tmem_ld_wait();
            if (c + 2 < nc) tmem_ld_x32(ts + 32 * c + 64, s0);
            row_exp(s1, nv - 32 * c - 32, c2, m2, sum, ts + 16 * c + 16);
          }
        }
        if (w.nt == 2) {
          if (lane == 0) mbar_arrive(&bars->order[t ^ 1][quarter]);
          ++turn;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->pready[t]);
        const float2 u0 = upk(sum[0]), u1 = upk(sum[1]);
        l += (u0.x + u0.y) + (u1.x + u1.y);
      }
      if (!ok) break;
      // the epilogue has read the last item's sums
      if (!(ok = warp_wait_near(&bars->ofree[t], (item & 1) ^ 1, abort_flag))) break;
      inv_l[t * BM + row] = l == 0.f ? 0.f : 1.f / l;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->lready[t]);
      ++item;
      const int64_t n = (int64_t(w.pair) * 2 + t) * BM + row;
      if (n < a.Nq) {
        const int64_t r = (int64_t(w.b) * a.H + w.h) * a.Nq + n;
        if (a.splits > 1)
          part_ml[int64_t(w.split) * a.rows + r] = make_float2(m * LN2, l);
        else if (lse)
          lse[r] = (m + __log2f(l)) * LN2;
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    regs_dec<REGS_EPI>();
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t item[2] = {0, 0};
    bool ok = true;
    for (int64_t i = blockIdx.x; ok && i < a.total; i += gridDim.x) {
      const Work w = get_work(a, i);
      for (int t = 0; t < w.nt; ++t) {
        const int64_t n = (int64_t(w.pair) * 2 + t) * BM + row;
        const int64_t r = (int64_t(w.b) * a.H + w.h) * a.Nq + n;
        __nv_bfloat16* o = O + w.b * a.o.b + w.h * a.o.h + n * a.o.n;
        float* po = part_o + (int64_t(w.split) * a.rows + r) * D;
        const bool in = n < a.Nq;
        float inv = 0.f;
        if (w.nk > 0) {
          ok = warp_wait_near(&bars->ofull[t], item[t] & 1, abort_flag) && warp_wait_near(&bars->lready[t], item[t] & 1, abort_flag);
          if (!ok) break;
          ++item[t];
          tc_fence_after();
          inv = inv_l[t * BM + row];
        } else if (in) {  // nothing attended: o = 0, lse = -inf
          if (a.splits > 1)
            part_ml[int64_t(w.split) * a.rows + r] = make_float2(xs::NEG_INF, 0.f);
          else if (lse)
            lse[r] = xs::NEG_INF;
        }
        const uint32_t ot = tmem + O_COL + 128u * t + lane_bits;
        // (by a loop: the kernel's code has to stay within the instruction cache)
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32] = {};
          if (w.nk > 0) {
            tmem_ld_x32(ot + 32 * c, v);
            tmem_ld_wait();
          }
          if (in) store_row32(o + 32 * c, po + 32 * c, v, a.splits > 1 ? 1.f : inv, a.splits > 1, wide != 0);
        }
        if (w.nk > 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->ofree[t]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) tmem_dealloc(tmem, 512);
}

}  // namespace xt
}  // namespace la
