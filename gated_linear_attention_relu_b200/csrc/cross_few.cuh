// cross_few.cuh -- cross attention forward of a few query rows (one new token per sequence, or a
// few, against long encoder states): all rows that read a key head, at most 8, in one block.
//
//   s_rj = scale q_r.k_j,  o_r = sum_j exp(s_rj - lse_r) v_j
//
// Bound by HBM: keys and values are read once for all rows together, 16 bytes a lane, a row of d
// channels by d * size / 16 neighbouring lanes.  A warp takes UNROLL * 2 (bf16, d = 128) keys at a
// time and keeps its own running maximum, sum and output.  Its next STAGES - 1 groups of keys are in
// flight to its part of shared memory meanwhile (each lane reads back what it copied itself, so
// nothing but the copies is waited for): loads into registers left the warp waiting for half of the
// time.  The block's warps are joined in shared memory in order, and the
// parts of the key axis (split over blocks: there are few heads) by join_kernel.  A tensor-core tile
// would be 128 rows for at most 8; the FMA pipe has the time: at 4 rows a key of 512 bytes costs
// about 46 instructions and its bytes about 88 issue slots.
// 8 x 8 key heads, 16384 keys, 4 rows each: 537 MB in 100 us (5.4 TB/s); lengths that leave half of the
// keys out 65 us, where the last wave's few blocks show.
#pragma once
#include "common.cuh"
#include "cross_simt.cuh"
#include "sm100.cuh"

namespace la {
namespace xf {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int UNROLL = 4;
constexpr int STAGES = 3;
constexpr uint32_t STAGE_BYTES = 2 * UNROLL * 32 * 16;  // of a warp: its lanes' keys, then values
constexpr int MAX_ROWS = 8;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

template <typename T, int CPL>
__device__ __forceinline__ void unpack2(const uint4& u, uint64_t (&f)[CPL / 2]) {
  if constexpr (CPL == 8) {
    f[0] = pk(bf16lo(u.x), bf16hi(u.x));
    f[1] = pk(bf16lo(u.y), bf16hi(u.y));
    f[2] = pk(bf16lo(u.z), bf16hi(u.z));
    f[3] = pk(bf16lo(u.w), bf16hi(u.w));
  } else {
    f[0] = pk(__uint_as_float(u.x), __uint_as_float(u.y));
    f[1] = pk(__uint_as_float(u.z), __uint_as_float(u.w));
  }
}

// Joins a value over the lanes that hold it for other keys (of the UNROLL, and of the other key
// groups of a load); every lane gets the result.
template <int LPK, typename F>
__device__ __forceinline__ float over_keys(float v, F&& f) {
  v = f(v, __shfl_xor_sync(0xffffffffu, v, LPK / 2));
  v = f(v, __shfl_xor_sync(0xffffffffu, v, LPK / 4));
#pragma unroll
  for (int o = LPK; o < 32; o <<= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
static_assert(UNROLL == 4, "over_keys");

template <int D, int R>
__host__ __device__ constexpr size_t smem_bytes() {
  return STAGES * WARPS * STAGE_BYTES > size_t(WARPS) * R * (D + 2) * 4 ? STAGES * WARPS * STAGE_BYTES
                                                                       : size_t(WARPS) * R * (D + 2) * 4;
}

// R: rows of the block (group * Nq of them used).
template <int D, typename T, int R>
__global__ void __launch_bounds__(THREADS, R <= 4 ? 2 : 1)
few_kernel(const __grid_constant__ xs::Args a, const T* __restrict__ Q, const T* __restrict__ K, const T* __restrict__ V,
           T* __restrict__ O, float* __restrict__ lse, float* __restrict__ part_o, float2* __restrict__ part_ml) {
  constexpr int CPL = 16 / int(sizeof(T));  // channels per lane
  constexpr int LPK = D / CPL;              // lanes per key
  constexpr int KPI = 32 / LPK;             // keys per load instruction
  constexpr int STEP = KPI * UNROLL;        // keys a warp takes at a time
  extern __shared__ __align__(16) float sm[];
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPK, ch = (lane % LPK) * CPL;
  const int64_t split = blockIdx.x % a.splits, hb = blockIdx.x / a.splits;
  const int64_t kh = hb % a.Hkv, b = hb / a.Hkv;
  const int rows = static_cast<int>(a.group * a.Nq);
  const int64_t limit = xs::key_limit(a, b);
  const int64_t k_begin = split * a.tiles_per_split * xs::BT;
  int64_t k_end = k_begin + int64_t(a.tiles_per_split) * xs::BT;
  if (k_end > limit) k_end = limit;
  const uint8_t* mask = a.mask ? a.mask + b * a.Nk : nullptr;

  // Scores k = u R + r of a key group, u of UNROLL and row r: lane i of a key's LPK lanes holds those
  // from (i / REP) CNT on.
  constexpr int NV = UNROLL * R;
  constexpr int CNT = NV > LPK ? NV / LPK : 1;
  constexpr int REP = NV < LPK ? LPK / NV : 1;
  const int k_own = (lane % LPK) / REP * CNT, u_own = k_own / R;
  uint64_t q[R][CPL / 2], acc[R][CPL / 2];
  float m[CNT], l[CNT];
#pragma unroll
  for (int i = 0; i < CNT; ++i) {
    m[i] = xs::LOWEST;
    l[i] = 0.f;
  }
  const float cexp = a.scale * LOG2E;
  const T* kb = K + b * a.k.b + kh * a.k.h + ch;
  const T* vb = V + b * a.v.b + kh * a.v.h + ch;
  const uint32_t ring = smem_u32(sm) + warp * (STAGES * STAGE_BYTES) + lane * 16;
  auto fetch = [&](int64_t j0, int stage) {
    if (j0 < k_end) {
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int64_t j = j0 + u * KPI + sub;
        const bool in = j < k_end;  // (else 0, and the address of the first key)
        const uint32_t at = ring + stage * STAGE_BYTES + u * 512;
        cp_async16(at, kb + (in ? j : k_begin) * a.k.n, in ? 16 : 0);
        cp_async16(at + UNROLL * 512, vb + (in ? j : k_begin) * a.v.n, in ? 16 : 0);
      }
    }
    cp_async_commit();
  };
  const int64_t j_first = k_begin + warp * STEP;
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(j_first + i * int64_t(WARPS * STEP), i);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int rr = r < rows ? r : 0;
    const int64_t h = kh * a.group + rr / a.Nq, n = rr % a.Nq;
    const uint4 u = *reinterpret_cast<const uint4*>(Q + b * a.q.b + h * a.q.h + n * a.q.n + ch);
    unpack2<T, CPL>(u, q[r]);
#pragma unroll
    for (int c = 0; c < CPL / 2; ++c) acc[r][c] = 0;
  }
  int stage = 0;
  for (int64_t j0 = j_first; j0 < k_end; j0 += WARPS * STEP) {
    fetch(j0 + (STAGES - 1) * int64_t(WARPS * STEP), stage == 0 ? STAGES - 1 : stage - 1);
    const int64_t j_own = j0 + u_own * KPI + sub;
    const bool ok = j_own < k_end && (!mask || mask[j_own] != 0);
    cp_async_wait<STAGES - 1>();
    const uint32_t at = ring + stage * STAGE_BYTES;
    if (++stage == STAGES) stage = 0;
    // a lane's share of every score ...
    float s[NV];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      uint64_t k2[CPL / 2];
      unpack2<T, CPL>(lds128(at + u * 512), k2);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        uint64_t t = mul2(q[r][0], k2[0]);
#pragma unroll
        for (int c = 1; c < CPL / 2; ++c) t = fma2(q[r][c], k2[c], t);
        const float2 f = upk(t);
        s[u * R + r] = f.x + f.y;
      }
    }
    // ... summed over the key's lanes, each of which ends up with CNT of the NV scores
    int cnt = NV;
#pragma unroll
    for (int o = LPK / 2; o > 0; o >>= 1) {
      if (cnt > 1) {
        cnt >>= 1;
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < NV / 2; ++i)
          if (i < cnt) {
            const float send = up ? s[i] : s[i + cnt], keep = up ? s[i + cnt] : s[i];
            s[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
          }
      } else {
        s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
      }
    }
    float top[CNT];
    bool raise = false;
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      if (!ok) s[i] = xs::NEG_INF;
      top[i] = over_keys<LPK>(s[i], [](float x, float y) { return fmaxf(x, y); });
      raise |= top[i] > m[i];
    }
    if (__any_sync(0xffffffffu, raise)) {
      float f[CNT];
#pragma unroll
      for (int i = 0; i < CNT; ++i) {
        top[i] = fmaxf(top[i], m[i]);
        f[i] = exp2_approx((m[i] - top[i]) * cexp);
        m[i] = top[i];
        l[i] *= f[i];
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float fr = __shfl_sync(0xffffffffu, f[r % CNT], (r / CNT) * REP, LPK);
#pragma unroll
        for (int c = 0; c < CPL / 2; ++c) acc[r][c] = mul2(acc[r][c], pk(fr, fr));
      }
    }
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      s[i] = ok ? exp2_approx((s[i] - m[i]) * cexp) : 0.f;
      l[i] += s[i];
    }
    const uint32_t all = mask ? __ballot_sync(0xffffffffu, ok) : 0xffffffffu;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      uint4 vu = lds128(at + (UNROLL + u) * 512);
      // whatever an unattended row holds has no influence
      if (all != 0xffffffffu && !((all >> (sub * LPK + (u * R / CNT) * REP)) & 1u)) vu = make_uint4(0, 0, 0, 0);
      uint64_t v2[CPL / 2];
      unpack2<T, CPL>(vu, v2);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int k = u * R + r;
        const float p = __shfl_sync(0xffffffffu, s[k % CNT], (k / CNT) * REP, LPK);
#pragma unroll
        for (int c = 0; c < CPL / 2; ++c) acc[r][c] = fma2(pk(p, p), v2[c], acc[r][c]);
      }
    }
  }
  // join the lanes that held different keys, then the warps (over the ring)
  cp_async_wait<0>();
  __syncthreads();
  float* sm_o = sm;                       // [WARPS][R][D]
  float* sm_ml = sm + WARPS * R * D;      // [WARPS][R][2]
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float o[CPL];
#pragma unroll
    for (int c = 0; c < CPL / 2; ++c) {
      const float2 f = upk(acc[r][c]);
      o[2 * c] = f.x;
      o[2 * c + 1] = f.y;
    }
#pragma unroll
    for (int d = LPK; d < 32; d <<= 1) {
#pragma unroll
      for (int c = 0; c < CPL; ++c) o[c] += __shfl_xor_sync(0xffffffffu, o[c], d);
    }
    if (sub == 0) {
#pragma unroll
      for (int c = 0; c < CPL; ++c) sm_o[(warp * R + r) * D + ch + c] = o[c];
    }
  }
#pragma unroll
  for (int i = 0; i < CNT; ++i) {
    l[i] = over_keys<LPK>(l[i], [](float x, float y) { return x + y; });
    if (sub == 0 && u_own == 0) {  // (lanes with the same row write the same values)
      sm_ml[(warp * R + k_own + i) * 2] = m[i];
      sm_ml[(warp * R + k_own + i) * 2 + 1] = l[i];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < rows * D; e += THREADS) {
    const int r = e / D, c = e % D;
    float M = xs::LOWEST;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm_ml[(w * R + r) * 2]);
    float L = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = exp2_approx((sm_ml[(w * R + r) * 2] - M) * cexp);
      L += f * sm_ml[(w * R + r) * 2 + 1];
      o += f * sm_o[(w * R + r) * D + c];
    }
    const int64_t h = kh * a.group + r / a.Nq, n = r % a.Nq;
    const int64_t row = (b * a.H + h) * a.Nq + n;
    if (a.splits > 1) {
      part_o[(split * a.rows + row) * D + c] = o;
      if (c == 0) part_ml[split * a.rows + row] = make_float2(M * a.scale, L);
    } else {
      ln::put(O[b * a.o.b + h * a.o.h + n * a.o.n + c], L == 0.f ? 0.f : o / L);
      if (lse && c == 0) lse[row] = L == 0.f ? xs::NEG_INF : M * a.scale + logf(L);
    }
  }
}

}  // namespace xf
}  // namespace la
