// cross_simt.cuh -- cross attention on the CUDA cores: fp32, and the reference point the
// tensor-core kernels are measured against (LA_FLAG_FORCE_SIMT).
//
//   s_ij = scale q_i.k_j,  o_i = sum_j exp(s_ij - lse_i) v_j   (la_cross_forward / _backward)
//
// One pass over the keys with the running maximum and sum of the softmax; 64 x 64 score tiles,
// 4 x 4 scores a thread, so a step along d feeds 16 FMAs from 8 shared-memory values; tiles of global
// memory are fetched into registers during the products of the tile before.  8 heads, 2048 x 1000,
// d = 128: forward 317 us (26 of 74.5 TFLOP/s), gradients 896 (23 in 5 products, 33 in the 7 done):
// the barriers between a tile's products and its exponentials leave the FMA pipe idle for the rest.
// Products over many keys (or, in the gradients, many queries) are summed
// per tile and the tiles' sums then added up, which keeps the rounding of long sums at the level of
// one tile.  Where there are too few tiles to fill the machine the long axis is split over blocks,
// whose partial results are joined in order by a second kernel.
#pragma once
#include "common.cuh"
#include "sm100.cuh"
#include "norm.cuh"

namespace la {
namespace xs {

constexpr int THREADS = 256;
constexpr int BT = 64;           // queries and keys per tile
constexpr int PS = BT + 4;       // row stride (floats) of a score tile
constexpr float NEG_INF = -__builtin_huge_valf();
// A running maximum to start from: -inf minus it is -inf and not NaN, so that scores of -inf weigh 0.
constexpr float LOWEST = -3.402823466e38f;

struct Str {
  int64_t b, h, n;
};

struct Args {
  int64_t B, H, Hkv, Nq, Nk;
  int64_t q_tiles, k_tiles;   // tiles of 64 per head
  int64_t rows;               // B * H * Nq
  int32_t group;              // H / Hkv
  int32_t splits, tiles_per_split;
  float scale;
  Str q, k, v, o, dout, dq, dk, dv;
  const int32_t* kv_len;
  const uint8_t* mask;
};

__device__ __forceinline__ int64_t key_limit(const Args& a, int64_t b) {
  if (!a.kv_len) return a.Nk;
  const int64_t n = a.kv_len[b];
  return n < 0 ? 0 : (n < a.Nk ? n : a.Nk);
}

template <int D>
__host__ __device__ constexpr int row_stride() { return D + 4; }  // floats: 16-byte rows whose float4 columns spread over the banks

// 64 rows of D channels on their way to shared memory: fetch() starts the loads (rows outside [0,
// valid) become 0 and are not read), stash() puts them there as fp32.  What is fetched before a tile's
// products and stashed after them costs no waiting.
template <int D, typename T>
struct Tile {
  static constexpr int VEC = 16 / int(sizeof(T)), PR = D / VEC, N = BT * PR / THREADS;
  ln::Pack<T, VEC> p[N];

  __device__ __forceinline__ void fetch(const T* src, int64_t stride, int valid) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int e = threadIdx.x + k * THREADS, r = e / PR;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (r < valid) u = __ldg(reinterpret_cast<const uint4*>(src + r * stride + (e % PR) * VEC));
      p[k] = *reinterpret_cast<const ln::Pack<T, VEC>*>(&u);
    }
  }
  __device__ __forceinline__ void stash(float* dst) const {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int e = threadIdx.x + k * THREADS;
      float* to = dst + e / PR * row_stride<D>() + (e % PR) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; i += 4)
        *reinterpret_cast<float4*>(to + i) = make_float4(p[k].get(i), p[k].get(i + 1), p[k].get(i + 2), p[k].get(i + 3));
    }
  }
};
template <int D, typename T>
__device__ __forceinline__ void load_tile(float* dst, const T* src, int64_t stride, int valid) {
  Tile<D, T> t;
  t.fetch(src, stride, valid);
  t.stash(dst);
}

// s[ii][jj] = A[ty + 16 ii] . B[tx + 16 jj]
template <int D>
__device__ __forceinline__ void mm_nt(const float* A, const float* B, int ty, int tx, float (&s)[4][4]) {
  uint64_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0;
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    ulonglong2 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const ulonglong2*>(A + (ty + 16 * i) * row_stride<D>() + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const ulonglong2*>(B + (tx + 16 * j) * row_stride<D>() + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fma2(x[i].x, y[j].x, acc[i][j]);
        acc[i][j] = fma2(x[i].y, y[j].y, acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 t = upk(acc[i][j]);
      s[i][j] = t.x + t.y;
    }
}

// Channel of pair k (of D / 32) of a thread: float4 columns where D has them, else float2.
template <int D>
__device__ __forceinline__ int chan(int tx, int k) {
  return D >= 64 ? 4 * tx + 64 * (k >> 1) + 2 * (k & 1) : 2 * tx;
}

// t[ii][k] = sum_j P[ty + 16 ii][j] B[j][chan(k)], j over the tile's 64 rows.
template <int D>
__device__ __forceinline__ void mm_nn(const float* P, const float* B, int ty, int tx, uint64_t (&t)[4][D / 32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < D / 32; ++k) t[i][k] = 0;
#pragma unroll 2
  for (int j = 0; j < BT; j += 4) {
    float4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty + 16 * i) * PS + j);
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      uint64_t b[D / 32];
      const float* row = B + (j + jj) * row_stride<D>();
      if constexpr (D >= 64) {
#pragma unroll
        for (int k = 0; k < D / 32; k += 2) {
          const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(row + chan<D>(tx, k));
          b[k] = u.x;
          b[k + 1] = u.y;
        }
      } else {
        b[0] = *reinterpret_cast<const uint64_t*>(row + chan<D>(tx, 0));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = jj == 0 ? p[i].x : (jj == 1 ? p[i].y : (jj == 2 ? p[i].z : p[i].w));
        const uint64_t vv = pk(v, v);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) t[i][k] = fma2(vv, b[k], t[i][k]);
      }
    }
  }
}

__device__ __forceinline__ float lane16_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float lane16_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D, typename T>
__device__ __forceinline__ void store_pair(T* dst, float2 v) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16(v.x, v.y);
  else
    *reinterpret_cast<float2*>(dst) = v;
}

// Block -> (tile, split, head): tiles fastest, so that neighbouring blocks read the same keys.
struct Where {
  int64_t tile, b, h;
  int split;
};
__device__ __forceinline__ Where where(const Args& a, int64_t tiles, int64_t heads) {
  Where w;
  int64_t i = blockIdx.x;
  w.tile = i % tiles;
  i /= tiles;
  w.split = static_cast<int>(i % a.splits);
  i /= a.splits;
  w.h = i % heads;
  w.b = i / heads;
  return w;
}

template <int D>
__host__ __device__ constexpr size_t fwd_smem() { return (2 * BT * row_stride<D>() + BT * PS) * 4; }

// Forward.  part_o [splits][rows][D] (sums over the split's keys) and part_ml [splits][rows] (the
// split's maximum and sum) when splits > 1, else O and lse themselves.
template <int D, typename T>
__global__ void __launch_bounds__(THREADS)
forward_kernel(const __grid_constant__ Args a, const T* __restrict__ Q, const T* __restrict__ K,
               const T* __restrict__ V, T* __restrict__ O, float* __restrict__ lse, float* __restrict__ part_o,
               float2* __restrict__ part_ml) {
  extern __shared__ __align__(16) float sm[];
  float* qs = sm;
  float* kv = qs + BT * row_stride<D>();
  float* ps = kv + BT * row_stride<D>();
  pdl_trigger();
  const Where w = where(a, a.q_tiles, a.H);
  const int64_t kh = w.h / a.group, q0 = w.tile * BT;
  const int qn = static_cast<int>(a.Nq - q0 < BT ? a.Nq - q0 : BT);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  pdl_wait();  // (gathered keys and their counts)
  const int64_t limit = key_limit(a, w.b);
  const int64_t k_begin = int64_t(w.split) * a.tiles_per_split * BT;
  int64_t k_end = k_begin + int64_t(a.tiles_per_split) * BT;
  if (k_end > limit) k_end = limit;

  load_tile<D>(qs, Q + w.b * a.q.b + w.h * a.q.h + q0 * a.q.n, a.q.n, qn);
  float m[4], l[4];
  uint64_t acc[4][D / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = NEG_INF;
    l[i] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) acc[i][k] = 0;
  }
  // (at D = 128 a second tile of registers would leave one block an SM)
  Tile<D, T> next;
  const T* kb = K + w.b * a.k.b + kh * a.k.h;
  const T* vb = V + w.b * a.v.b + kh * a.v.h;
  if (k_begin < k_end) next.fetch(kb + k_begin * a.k.n, a.k.n, static_cast<int>(k_end - k_begin < BT ? k_end - k_begin : BT));
  for (int64_t k0 = k_begin; k0 < k_end; k0 += BT) {
    const int kn = static_cast<int>(k_end - k0 < BT ? k_end - k0 : BT);
    next.stash(kv);
    __syncthreads();
    next.fetch(vb + k0 * a.v.n, a.v.n, kn);
    float s[4][4];
    mm_nt<D>(qs, kv, ty, tx, s);
    float corr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = NEG_INF;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = tx + 16 * j < kn ? s[i][j] * a.scale : NEG_INF;
        mx = fmaxf(mx, s[i][j]);
      }
      const float m_new = fmaxf(m[i], lane16_max(mx));
      const float m_use = m_new == NEG_INF ? 0.f : m_new;  // nothing attended so far
      corr[i] = m[i] == NEG_INF ? 0.f : expf(m[i] - m_use);
      m[i] = m_new;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = s[i][j] == NEG_INF ? 0.f : expf(s[i][j] - m_use);
        sum += p;
        ps[(ty + 16 * i) * PS + tx + 16 * j] = p;
      }
      l[i] = l[i] * corr[i] + lane16_sum(sum);
    }
    __syncthreads();  // the keys have been read
    next.stash(kv);
    __syncthreads();
    const int64_t k1 = k0 + BT;
    if (k1 < k_end) next.fetch(kb + k1 * a.k.n, a.k.n, static_cast<int>(k_end - k1 < BT ? k_end - k1 : BT));
    uint64_t t[4][D / 32];
    mm_nn<D>(ps, kv, ty, tx, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t c2 = pk(corr[i], corr[i]);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) acc[i][k] = fma2(acc[i][k], c2, t[i][k]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i;
    if (r >= qn) continue;
    const int64_t row = (w.b * a.H + w.h) * a.Nq + q0 + r;
    if (a.splits > 1) {
      const int64_t slot = int64_t(w.split) * a.rows + row;
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
        *reinterpret_cast<float2*>(part_o + slot * D + chan<D>(tx, k)) = upk(acc[i][k]);
      if (tx == 0) part_ml[slot] = make_float2(m[i], l[i]);
    } else {
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];  // (a sum of NaN stays one)
      T* o = O + w.b * a.o.b + w.h * a.o.h + (q0 + r) * a.o.n;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const float2 v = upk(acc[i][k]);
        store_pair<D>(o + chan<D>(tx, k), make_float2(v.x * inv, v.y * inv));
      }
      if (lse && tx == 0) lse[row] = l[i] == 0.f ? NEG_INF : m[i] + logf(l[i]);
    }
  }
}

// Joins the splits' partial results, one block per row: with M the largest maximum,
// o = sum_s e^(m_s - M) o_s / sum_s e^(m_s - M) l_s.  A warp adds every JOIN_WARPS-th part, and the
// warps' sums are added in order.
constexpr int JOIN_WARPS = 4, MAX_SPLITS = 1024;

template <int D, typename T>
__global__ void __launch_bounds__(32 * JOIN_WARPS)
join_kernel(const __grid_constant__ Args a, const float* __restrict__ part_o, const float2* __restrict__ part_ml,
            T* __restrict__ O, float* __restrict__ lse) {
  __shared__ float f[MAX_SPLITS];
  __shared__ float red[JOIN_WARPS], sums[JOIN_WARPS][D];
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float top = NEG_INF;
  for (int s = threadIdx.x; s < a.splits; s += 32 * JOIN_WARPS) {
    f[s] = part_ml[int64_t(s) * a.rows + row].x;
    top = fmaxf(top, f[s]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) red[warp] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float M = top == NEG_INF ? 0.f : top;  // (nothing attended: every factor is 0)
  __syncthreads();
  float L = 0.f;
  for (int s = threadIdx.x; s < a.splits; s += 32 * JOIN_WARPS) {
    const float l = part_ml[int64_t(s) * a.rows + row].y;
    f[s] = l == 0.f ? 0.f : expf(f[s] - M);
    L += f[s] * l;
  }
  L = ln::warp_sum(L);
  if (lane == 0) red[warp] = L;
  __syncthreads();
  L = (red[0] + red[1]) + (red[2] + red[3]);
  constexpr int C = D / 32;
  float acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
  const float* po = part_o + row * D + lane;
  int s = warp;
  for (; s + 7 * JOIN_WARPS < a.splits; s += 8 * JOIN_WARPS) {  // (a part without keys has sums of 0)
    float v[8][C];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int c = 0; c < C; ++c) v[k][c] = po[int64_t(s + k * JOIN_WARPS) * a.rows * D + 32 * c];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] += f[s + k * JOIN_WARPS] * v[k][c];
  }
  for (; s < a.splits; s += JOIN_WARPS)
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] += f[s] * po[int64_t(s) * a.rows * D + 32 * c];
#pragma unroll
  for (int c = 0; c < C; ++c) sums[warp][lane + 32 * c] = acc[c];
  __syncthreads();
  const int64_t n = row % a.Nq, bh = row / a.Nq;
  T* o = O + (bh / a.H) * a.o.b + (bh % a.H) * a.o.h + n * a.o.n;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  for (int c = threadIdx.x; c < D; c += 32 * JOIN_WARPS)
    ln::put(o[c], ((sums[0][c] + sums[1][c]) + (sums[2][c] + sums[3][c])) * inv);
  if (lse && threadIdx.x == 0) lse[row] = L == 0.f ? NEG_INF : M + logf(L);
}

// D_i = dO_i . O_i for every query row.  A block has consecutive rows of a head; a row belongs to
// D * size / 16 neighbouring lanes, and DELTA_ROWS rows of each lane are in flight.
constexpr int DELTA_ROWS = 8;
template <int D, typename T>
__host__ __device__ constexpr int delta_rows() { return THREADS / (D * int(sizeof(T)) / 16) * DELTA_ROWS; }  // per block

template <int D, typename T>
__global__ void __launch_bounds__(THREADS)
delta_kernel(const __grid_constant__ Args a, const T* __restrict__ O, const T* __restrict__ dO, float* __restrict__ delta) {
  constexpr int VEC = 16 / int(sizeof(T)), LPR = D / VEC, STEP = THREADS / LPR;
  pdl_trigger();
  pdl_wait();  // (it reads nothing of the gather's, but the kernels after it wait for this one only)
  const uint32_t tiles = static_cast<uint32_t>((a.Nq + delta_rows<D, T>() - 1) / delta_rows<D, T>());
  const uint32_t bh = blockIdx.x / tiles, b = bh / static_cast<uint32_t>(a.H), h = bh - b * static_cast<uint32_t>(a.H);
  const int64_t n0 = int64_t(blockIdx.x - bh * tiles) * delta_rows<D, T>() + threadIdx.x / LPR;
  const int c = (threadIdx.x % LPR) * VEC;
  const T* po = O + b * a.o.b + h * a.o.h + n0 * a.o.n + c;
  const T* pg = dO + b * a.dout.b + h * a.dout.h + n0 * a.dout.n + c;
  ln::Pack<T, VEC> o[DELTA_ROWS], g[DELTA_ROWS];
#pragma unroll
  for (int k = 0; k < DELTA_ROWS; ++k)
    if (n0 + k * STEP < a.Nq) {
      o[k] = *reinterpret_cast<const ln::Pack<T, VEC>*>(po + int64_t(k) * STEP * a.o.n);
      g[k] = *reinterpret_cast<const ln::Pack<T, VEC>*>(pg + int64_t(k) * STEP * a.dout.n);
    }
#pragma unroll
  for (int k = 0; k < DELTA_ROWS; ++k) {
    const int64_t n = n0 + k * STEP;
    float s = 0.f;
    if (n < a.Nq)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += o[k].get(e) * g[k].get(e);
    s = ln::lanes_sum<LPR>(s);
    if (n < a.Nq && c == 0) delta[bh * a.Nq + n] = s;
  }
}

template <int D>
__host__ __device__ constexpr size_t bwd_smem() { return (4 * BT * row_stride<D>() + BT * PS + 2 * BT) * 4; }

// The gradients' threads: a warp covers 4 x 8 of the 16 x 16, so that each of a step's shared-memory
// loads is one wavefront (2 x 16, which the forward's row sums want, takes 12 instead of 8 for the
// scores' 16 cycles of FMAs).
__device__ __forceinline__ void thread_tile(int& tx, int& ty) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  tx = (warp & 1) * 8 + (lane & 7);
  ty = (warp >> 1) * 4 + (lane >> 3);
}

// dQ of one query tile over the split's keys; part [splits][rows][D] when splits > 1.
template <int D, typename T>
__global__ void __launch_bounds__(THREADS)
dq_kernel(const __grid_constant__ Args a, const T* __restrict__ Q, const T* __restrict__ K, const T* __restrict__ V,
          const T* __restrict__ dO, const float* __restrict__ lse, const float* __restrict__ delta,
          T* __restrict__ dQ, float* __restrict__ part) {
  extern __shared__ __align__(16) float sm[];
  constexpr int RS = row_stride<D>();
  float* qs = sm;
  float* gs = qs + BT * RS;
  float* ks = gs + BT * RS;
  float* vs = ks + BT * RS;
  float* ps = vs + BT * RS;
  pdl_trigger();
  const Where w = where(a, a.q_tiles, a.H);
  const int64_t kh = w.h / a.group, q0 = w.tile * BT;
  const int qn = static_cast<int>(a.Nq - q0 < BT ? a.Nq - q0 : BT);
  int tx, ty;
  thread_tile(tx, ty);
  pdl_wait();  // D_i, gathered keys and their counts
  const int64_t limit = key_limit(a, w.b);
  const int64_t k_begin = int64_t(w.split) * a.tiles_per_split * BT;
  int64_t k_end = k_begin + int64_t(a.tiles_per_split) * BT;
  if (k_end > limit) k_end = limit;
  const int64_t row0 = (w.b * a.H + w.h) * a.Nq + q0;

  load_tile<D>(qs, Q + w.b * a.q.b + w.h * a.q.h + q0 * a.q.n, a.q.n, qn);
  load_tile<D>(gs, dO + w.b * a.dout.b + w.h * a.dout.h + q0 * a.dout.n, a.dout.n, qn);
  float L[4], dl[4];
  uint64_t acc[4][D / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i;
    L[i] = r < qn ? lse[row0 + r] : 0.f;
    dl[i] = r < qn ? delta[row0 + r] : 0.f;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) acc[i][k] = 0;
  }
  Tile<D, T> tk, tv;
  const T* kb = K + w.b * a.k.b + kh * a.k.h;
  const T* vb = V + w.b * a.v.b + kh * a.v.h;
  auto fetch = [&](int64_t k0) {
    if (k0 >= k_end) return;
    const int kn = static_cast<int>(k_end - k0 < BT ? k_end - k0 : BT);
    tk.fetch(kb + k0 * a.k.n, a.k.n, kn);
    tv.fetch(vb + k0 * a.v.n, a.v.n, kn);
  };
  fetch(k_begin);
  for (int64_t k0 = k_begin; k0 < k_end; k0 += BT) {
    const int kn = static_cast<int>(k_end - k0 < BT ? k_end - k0 : BT);
    __syncthreads();
    tk.stash(ks);
    tv.stash(vs);
    __syncthreads();
    fetch(k0 + BT);
    float s[4][4], dp[4][4];
    mm_nt<D>(qs, ks, ty, tx, s);
    mm_nt<D>(gs, vs, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = tx + 16 * j < kn ? expf(s[i][j] * a.scale - L[i]) : 0.f;
        ps[(ty + 16 * i) * PS + tx + 16 * j] = p * (dp[i][j] - dl[i]) * a.scale;
      }
    __syncthreads();
    uint64_t t[4][D / 32];
    mm_nn<D>(ps, ks, ty, tx, t);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < D / 32; ++k) acc[i][k] = add2(acc[i][k], t[i][k]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i;
    if (r >= qn) continue;
    T* o = dQ + w.b * a.dq.b + w.h * a.dq.h + (q0 + r) * a.dq.n;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const float2 v = upk(acc[i][k]);
      if (a.splits > 1)
        *reinterpret_cast<float2*>(part + (int64_t(w.split) * a.rows + row0 + r) * D + chan<D>(tx, k)) = v;
      else
        store_pair<D>(o + chan<D>(tx, k), v);
    }
  }
}

// dK and dV of one key tile over the split's query tiles (all heads of the group, head after head);
// part_k, part_v [splits][B * Hkv * Nk][D] where given (else dK and dV themselves; splits = 1).
template <int D, typename T>
__global__ void __launch_bounds__(THREADS)
dkv_kernel(const __grid_constant__ Args a, const T* __restrict__ Q, const T* __restrict__ K, const T* __restrict__ V,
           const T* __restrict__ dO, const float* __restrict__ lse, const float* __restrict__ delta,
           T* __restrict__ dK, T* __restrict__ dV, float* __restrict__ part_k, float* __restrict__ part_v) {
  extern __shared__ __align__(16) float sm[];
  constexpr int RS = row_stride<D>();
  float* qs = sm;
  float* gs = qs + BT * RS;
  float* ks = gs + BT * RS;
  float* vs = ks + BT * RS;
  float* ps = vs + BT * RS;
  float* ls = ps + BT * PS;
  float* ds = ls + BT;
  pdl_trigger();
  const Where w = where(a, a.k_tiles, a.Hkv);
  const int64_t k0 = w.tile * BT;
  const int kn = static_cast<int>(a.Nk - k0 < BT ? a.Nk - k0 : BT);
  int tx, ty;
  thread_tile(tx, ty);
  pdl_wait();  // D_i, gathered keys and their counts
  const int64_t limit = key_limit(a, w.b);
  const int attended = limit - k0 < kn ? (limit > k0 ? static_cast<int>(limit - k0) : 0) : kn;
  load_tile<D>(ks, K + w.b * a.k.b + w.h * a.k.h + k0 * a.k.n, a.k.n, attended);
  load_tile<D>(vs, V + w.b * a.v.b + w.h * a.v.h + k0 * a.v.n, a.v.n, attended);
  uint64_t ak[4][D / 32], av[4][D / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < D / 32; ++k) ak[i][k] = av[i][k] = 0;
  const int64_t tiles = a.q_tiles * a.group;
  const int64_t t0 = int64_t(w.split) * a.tiles_per_split;
  int64_t t1 = t0 + a.tiles_per_split;
  if (t1 > tiles) t1 = tiles;
  if (k0 >= limit) t1 = t0;  // no key of this tile is attended
  Tile<D, T> tq, tg;
  float l_next = 0.f, d_next = 0.f;
  auto fetch = [&](int64_t it) {
    if (it >= t1) return;
    const int64_t h = w.h * a.group + it / a.q_tiles, q0 = (it % a.q_tiles) * BT;
    const int qn = static_cast<int>(a.Nq - q0 < BT ? a.Nq - q0 : BT);
    tq.fetch(Q + w.b * a.q.b + h * a.q.h + q0 * a.q.n, a.q.n, qn);
    tg.fetch(dO + w.b * a.dout.b + h * a.dout.h + q0 * a.dout.n, a.dout.n, qn);
    if (int(threadIdx.x) < qn) {
      const int64_t row = (w.b * a.H + h) * a.Nq + q0 + threadIdx.x;
      l_next = lse[row];
      d_next = delta[row];
    }
  };
  fetch(t0);
  for (int64_t it = t0; it < t1; ++it) {
    const int64_t q0 = (it % a.q_tiles) * BT;
    const int qn = static_cast<int>(a.Nq - q0 < BT ? a.Nq - q0 : BT);
    __syncthreads();
    tq.stash(qs);
    tg.stash(gs);
    if (threadIdx.x < BT) {
      ls[threadIdx.x] = l_next;
      ds[threadIdx.x] = d_next;
    }
    __syncthreads();
    fetch(it + 1);
    float s[4][4], dp[4][4];
    mm_nt<D>(ks, qs, ty, tx, s);   // s[key][query]
    mm_nt<D>(vs, gs, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = tx + 16 * j;
        const float p = (ty + 16 * i < attended && c < qn) ? expf(s[i][j] * a.scale - ls[c]) : 0.f;
        s[i][j] = p * (dp[i][j] - ds[c]) * a.scale;
        ps[(ty + 16 * i) * PS + c] = p;
      }
    __syncthreads();
    uint64_t t[4][D / 32];
    mm_nn<D>(ps, gs, ty, tx, t);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < D / 32; ++k) av[i][k] = add2(av[i][k], t[i][k]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) ps[(ty + 16 * i) * PS + tx + 16 * j] = s[i][j];
    __syncthreads();
    mm_nn<D>(ps, qs, ty, tx, t);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < D / 32; ++k) ak[i][k] = add2(ak[i][k], t[i][k]);
  }
  const int64_t keys = a.B * a.Hkv * a.Nk;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty + 16 * i;
    if (r >= kn) continue;
    const int64_t key = (w.b * a.Hkv + w.h) * a.Nk + k0 + r;
    T* ok_ = dK + w.b * a.dk.b + w.h * a.dk.h + (k0 + r) * a.dk.n;
    T* ov = dV + w.b * a.dv.b + w.h * a.dv.h + (k0 + r) * a.dv.n;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const int c = chan<D>(tx, k);
      if (part_k) {
        const int64_t at = (int64_t(w.split) * keys + key) * D + c;
        *reinterpret_cast<float2*>(part_k + at) = upk(ak[i][k]);
        *reinterpret_cast<float2*>(part_v + at) = upk(av[i][k]);
      } else {
        store_pair<D>(ok_ + c, upk(ak[i][k]));
        store_pair<D>(ov + c, upk(av[i][k]));
      }
    }
  }
}

// dQ: out[b, h, n] = sum over the splits, in order, of part[s][(b * H + h) * Nq + n]; one thread per
// pair of channels.
template <int D, typename T>
__global__ void __launch_bounds__(THREADS)
sum_rows_kernel(const __grid_constant__ Args a, const float* __restrict__ part, T* __restrict__ dQ) {
  pdl_wait();
  const int64_t e = int64_t(blockIdx.x) * THREADS + threadIdx.x;
  const int64_t row = e / (D / 2);
  const int c = static_cast<int>(e % (D / 2)) * 2;
  if (row >= a.rows) return;
  float2 v = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const float2 u = *reinterpret_cast<const float2*>(part + (int64_t(s) * a.rows + row) * D + c);
    v.x += u.x;
    v.y += u.y;
  }
  const int64_t n = row % a.Nq, bh = row / a.Nq;
  store_pair<D>(dQ + (bh / a.H) * a.dq.b + (bh % a.H) * a.dq.h + n * a.dq.n + c, v);
}

// dK and dV from the parts' sums, in order: key j of (b, h) is row place[b][j] of the parts (j itself
// when nothing was gathered; 0 where it is not attended).  A thread has 2 channels; blockIdx.y
// selects dK or dV.
template <int D, typename T>
__global__ void __launch_bounds__(THREADS)
sum_keys_kernel(int64_t keys, int64_t Hkv, int64_t Nk, int splits, const float* __restrict__ part_k,
                const float* __restrict__ part_v, const int32_t* __restrict__ place, T* __restrict__ dK,
                T* __restrict__ dV, Str sk, Str sv) {
  pdl_wait();
  const int64_t e = int64_t(blockIdx.x) * THREADS + threadIdx.x;
  const int64_t key = e / (D / 2);
  const int c = static_cast<int>(e % (D / 2)) * 2;
  if (key >= keys) return;
  const int64_t n = key % Nk, bh = key / Nk, b = bh / Hkv;
  const float* part = blockIdx.y == 0 ? part_k : part_v;
  const Str st = blockIdx.y == 0 ? sk : sv;
  T* out = (blockIdx.y == 0 ? dK : dV) + b * st.b + (bh % Hkv) * st.h + n * st.n + c;
  const int64_t at = place ? int64_t(place[b * Nk + n]) : n;
  float2 v = make_float2(0.f, 0.f);
  if (at >= 0) {
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float2 u = *reinterpret_cast<const float2*>(part + (int64_t(s) * keys + bh * Nk + at) * D + c);
      v.x += u.x;
      v.y += u.y;
    }
  }
  store_pair<D>(out, v);
}

// Gathers the attended keys: kc, vc [B, Hkv, pad, D] hold the rows of K and V that are attended, in
// order, then zeros up to a multiple of 16 rows (what lies behind is never read); count[b] is their
// number and place[b][j] where key j went (-1: unattended).  Unattended rows are not read.
// One block per 64 keys, head and batch row; each counts the attended keys before its own
// (of the mask; where Nk is long, of the sums that count_kernel took over G_SPAN keys each, and of the
// rest of the mask).
constexpr int G_THREADS = 256, G_KEYS = 64, G_SPAN = 4096;

// spans[b][i] = attended keys among keys [G_SPAN i, G_SPAN (i + 1)) of batch row b.
__global__ void __launch_bounds__(G_THREADS)
count_kernel(int64_t Nk, const int32_t* __restrict__ kv_len, const uint8_t* __restrict__ mask, int32_t* __restrict__ spans) {
  __shared__ int part[G_THREADS / 32];
  pdl_trigger();
  const int64_t per_row = (Nk + G_SPAN - 1) / G_SPAN;
  const int64_t i = blockIdx.x % per_row, b = blockIdx.x / per_row;
  int64_t limit = Nk;
  if (kv_len) limit = kv_len[b] < 0 ? 0 : (kv_len[b] < Nk ? kv_len[b] : Nk);
  const int64_t end = (i + 1) * G_SPAN < limit ? (i + 1) * G_SPAN : limit;
  int n = 0;
  for (int64_t j = i * G_SPAN + threadIdx.x; j < end; j += G_THREADS) n += mask[b * Nk + j] != 0;
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = n;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int k = 1; k < G_THREADS / 32; ++k) n += part[k];
    spans[blockIdx.x] = n;
  }
}

// PR: 16-byte packs of a row of d channels.  Strides count elements of T.
template <typename T, int PR>
__global__ void __launch_bounds__(G_THREADS)
gather_kernel(int64_t Hkv, int64_t Nk, int64_t pad, const T* __restrict__ K, const T* __restrict__ V, Str sk, Str sv,
              const int32_t* __restrict__ kv_len, const uint8_t* __restrict__ mask, const int32_t* __restrict__ spans,
              T* __restrict__ kc, T* __restrict__ vc, int32_t* __restrict__ count, int32_t* __restrict__ place) {
  constexpr int VEC = 16 / int(sizeof(T)), D = PR * VEC;
  __shared__ int before[G_THREADS / 32];
  __shared__ int pos[G_KEYS];
  __shared__ int own[2];
  pdl_trigger();
  const int64_t chunks = (Nk + G_KEYS - 1) / G_KEYS;
  const int64_t chunk = blockIdx.x % chunks, hb = blockIdx.x / chunks;
  const int64_t h = hb % Hkv, b = hb / Hkv;
  int64_t limit = Nk;
  if (kv_len) limit = kv_len[b] < 0 ? 0 : (kv_len[b] < Nk ? kv_len[b] : Nk);
  const int64_t k0 = chunk * G_KEYS;
  const uint8_t* mb = mask ? mask + b * Nk : nullptr;
  const int64_t head = k0 < limit ? k0 : limit;
  int n = 0;
  if (mb) {
    int64_t from = 0;
    if (spans) {
      pdl_wait();
      from = k0 / G_SPAN * G_SPAN;
      const int32_t* sb = spans + b * ((Nk + G_SPAN - 1) / G_SPAN);
      for (int64_t i = threadIdx.x; i < k0 / G_SPAN; i += G_THREADS) n += sb[i];
    }
    for (int64_t j = from + threadIdx.x; j < head; j += G_THREADS) n += mb[j] != 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0) before[threadIdx.x >> 5] = n;
  } else if ((threadIdx.x & 31) == 0) {
    before[threadIdx.x >> 5] = threadIdx.x == 0 ? static_cast<int>(head) : 0;
  }
  bool at = false;
  uint32_t ball = 0;
  if (threadIdx.x < G_KEYS) {
    const int64_t j = k0 + threadIdx.x;
    at = j < limit && (!mb || mb[j] != 0);
    ball = __ballot_sync(0xffffffffu, at);
    if ((threadIdx.x & 31) == 0) own[threadIdx.x >> 5] = __popc(ball);
  }
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int i = 0; i < G_THREADS / 32; ++i) base += before[i];
  if (threadIdx.x < G_KEYS) {
    const int p = base + (threadIdx.x >= 32 ? own[0] : 0) + __popc(ball & ((1u << (threadIdx.x & 31)) - 1u));
    pos[threadIdx.x] = at ? p : -1;
    if (h == 0 && k0 + threadIdx.x < Nk) place[b * Nk + k0 + threadIdx.x] = at ? p : -1;
  }
  __syncthreads();
  const int64_t row0 = (b * Hkv + h) * pad;
  for (int e = threadIdx.x; e < G_KEYS * PR; e += G_THREADS) {
    const int r = e / PR, c = (e % PR) * VEC;
    if (pos[r] < 0) continue;
    const int64_t j = k0 + r, to = (row0 + pos[r]) * D + c;
    *reinterpret_cast<uint4*>(kc + to) = *reinterpret_cast<const uint4*>(K + b * sk.b + h * sk.h + j * sk.n + c);
    *reinterpret_cast<uint4*>(vc + to) = *reinterpret_cast<const uint4*>(V + b * sv.b + h * sv.h + j * sv.n + c);
  }
  if (chunk == chunks - 1) {
    const int total = base + own[0] + own[1];
    if (h == 0 && threadIdx.x == 0) count[b] = total;
    const int rows = ((total + 15) & ~15) - total;
    for (int e = threadIdx.x; e < rows * PR; e += G_THREADS) {
      const int64_t to = (row0 + total + e / PR) * D + (e % PR) * VEC;
      *reinterpret_cast<uint4*>(kc + to) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(vc + to) = make_uint4(0, 0, 0, 0);
    }
  }
}

}  // namespace xs
}  // namespace la
