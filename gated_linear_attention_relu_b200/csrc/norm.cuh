// norm.cuh -- layer norm over the last dimension, forward and backward (la_layernorm_*).
//
//   y = (x - mean) rstd w_g + b_g;   with xh = (x - mean) rstd and a = dy w_g:
//   dx = rstd (a - mean(a) - xh mean(a xh)),  dw_g = sum dy xh,  db_g = sum dy.
//
// Both are bound by HBM: one read of x (and dy), one write of y (dx).  A row stays in registers
// between its read and its write, so the variance is the exact two-pass one.  A row belongs to one
// warp where it fits (no barrier), else to a block.  In the backward pass a thread owns the same
// columns of every row it sees, so its shares of dw and db stay in registers until the block has
// walked its range of rows; blocks write them to their own slots, which a second kernel adds in
// order (no atomics: the same bits every time).
#pragma once
#include "common.cuh"
#include "sm100.cuh"

namespace la {
namespace ln {

// VEC elements of a row, as loaded: 16 bytes where rows are 16-byte aligned, else one element.
template <typename T, int VEC>
struct Pack {
  T v[VEC];
};
template <>
struct __align__(16) Pack<__nv_bfloat16, 8> {
  __nv_bfloat16 v[8];
};
template <>
struct __align__(16) Pack<float, 4> {
  float v[4];
};

__device__ __forceinline__ float as_f(float x) { return x; }
__device__ __forceinline__ float as_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float& d, float x) { d = x; }
__device__ __forceinline__ void put(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

template <int VEC>
__device__ __forceinline__ void load_w(const float* __restrict__ w, float (&o)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(w + i));
      o[i] = t.x; o[i + 1] = t.y; o[i + 2] = t.z; o[i + 3] = t.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = __ldg(w + i);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the WPR warps of a row, in warp order (a row of one warp needs no shared memory).
// `red` is used by one sum at a time: callers alternate between two buffers.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (WPR > 1) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[w] = v;
    __syncthreads();
    v = warp_sum(lane < WPR ? red[lane] : 0.f);
  }
  return v;
}

struct Args {
  int64_t rows, per_group, sx, sy, sdy, sdx;
  int32_t cols;
  float eps, inv_cols;
};

constexpr int WARP_ROWS = 4;  // rows (warps) per block where a row belongs to one warp

// Element offset of pack i of this thread (may be >= cols: then the pack is absent; cols is a
// multiple of VEC).
template <int VEC, int WPR>
__device__ __forceinline__ int col_of(int i) {
  const int t = WPR == 1 ? int(threadIdx.x & 31) : int(threadIdx.x);
  return (i * 32 * WPR + t) * VEC;
}

template <typename T, int VEC, int NV, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 32 * WARP_ROWS : 32 * WPR)
forward_kernel(const Args a, const T* x, const float* __restrict__ weight,
               const float* __restrict__ bias, T* y, float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float red[2][32];
  const int64_t row = WPR == 1 ? int64_t(blockIdx.x) * WARP_ROWS + (threadIdx.x >> 5) : int64_t(blockIdx.x);
  if (row >= a.rows) return;  // (whole warps; a block of one row never leaves here)
  const T* xr = x + row * a.sx;
  Pack<T, VEC> p[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = col_of<VEC, WPR>(i);
    if (c < a.cols) p[i] = *reinterpret_cast<const Pack<T, VEC>*>(xr + c);
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (col_of<VEC, WPR>(i) < a.cols) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += as_f(p[i].v[e]);
    }
  const float mu = row_sum<WPR>(s, red[0]) * a.inv_cols;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (col_of<VEC, WPR>(i) < a.cols) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = as_f(p[i].v[e]) - mu;
        s += d * d;
      }
    }
  const float r = 1.f / sqrtf(row_sum<WPR>(s, red[1]) * a.inv_cols + a.eps);
  if (mean && (WPR == 1 ? (threadIdx.x & 31) == 0 : threadIdx.x == 0)) {
    mean[row] = mu;
    rstd[row] = r;
  }
  const int64_t g = row / a.per_group * a.cols;
  T* yr = y + row * a.sy;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = col_of<VEC, WPR>(i);
    if (c >= a.cols) continue;
    float w[VEC], b[VEC];
    if (weight) load_w<VEC>(weight + g + c, w);
    if (bias) load_w<VEC>(bias + g + c, b);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float v = (as_f(p[i].v[e]) - mu) * r;
      if (weight) v *= w[e];
      if (bias) v += b[e];
      put(p[i].v[e], v);
    }
    *reinterpret_cast<Pack<T, VEC>*>(yr + c) = p[i];
  }
}

// Block `part` of group g walks the group's rows part, part + parts, ... and leaves its sums in
// slot g * parts + part of `slots` ([2][groups * parts][cols]: dw, db), or in dweight and dbias
// themselves when parts is 1.
template <typename T, int VEC, int NV, int WPR>
__global__ void __launch_bounds__(32 * (WPR == 1 ? WARP_ROWS : WPR))
backward_kernel(const Args a, int parts, const T* x, const T* dy, const float* __restrict__ weight,
                const float* __restrict__ mean, const float* __restrict__ rstd, T* dx, float* dw_out, float* db_out) {
  constexpr int STEP = WPR == 1 ? WARP_ROWS : 1;  // rows a block takes at a time
  __shared__ float2 red[2][32];
  extern __shared__ float cross[];  // rows of one warp each: the warps' sums, joined at the end
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t g = blockIdx.x / static_cast<uint32_t>(parts);
  const int part = static_cast<int>(blockIdx.x - g * parts);
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = col_of<VEC, WPR>(i);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[i][e] = 1.f;
      dw[i][e] = db[i][e] = 0.f;
    }
    if (weight && c < a.cols) load_w<VEC>(weight + g * a.cols + c, w[i]);
  }
  int buf = 0;
  for (int64_t j = int64_t(part) * STEP + (WPR == 1 ? warp : 0); j < a.per_group; j += int64_t(parts) * STEP) {
    const int64_t row = g * a.per_group + j;
    Pack<T, VEC> px[NV], pd[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col_of<VEC, WPR>(i);
      if (c < a.cols) {
        px[i] = *reinterpret_cast<const Pack<T, VEC>*>(x + row * a.sx + c);
        pd[i] = *reinterpret_cast<const Pack<T, VEC>*>(dy + row * a.sdy + c);
      }
    }
    const float mu = mean[row], r = rstd[row];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (col_of<VEC, WPR>(i) < a.cols) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (as_f(px[i].v[e]) - mu) * r, d = as_f(pd[i].v[e]);
          dw[i][e] += d * xh;
          db[i][e] += d;
          s1 += d * w[i][e];
          s2 += d * w[i][e] * xh;
        }
      }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if constexpr (WPR > 1) {
      if (lane == 0) red[buf][warp] = make_float2(s1, s2);
      __syncthreads();
      const float2 t = lane < WPR ? red[buf][lane] : make_float2(0.f, 0.f);
      s1 = warp_sum(t.x);
      s2 = warp_sum(t.y);
      buf ^= 1;  // the next row's sums go to the other buffer: one barrier per row is enough
    }
    const float c1 = s1 * a.inv_cols, c2 = s2 * a.inv_cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col_of<VEC, WPR>(i);
      if (c >= a.cols) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (as_f(px[i].v[e]) - mu) * r;
        put(px[i].v[e], r * (as_f(pd[i].v[e]) * w[i][e] - c1 - xh * c2));
      }
      *reinterpret_cast<Pack<T, VEC>*>(dx + row * a.sdx + c) = px[i];
    }
  }
  if (!dw_out && !db_out) return;
  const int64_t slot = int64_t(blockIdx.x) * a.cols;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* out = k == 0 ? dw_out : db_out;
    if (!out) continue;
    if constexpr (WPR == 1) {
      // the block's warps saw different rows of the same columns: join them in warp order
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = col_of<VEC, WPR>(i);
        if (c < a.cols)
#pragma unroll
          for (int e = 0; e < VEC; ++e) cross[warp * a.cols + c + e] = k == 0 ? dw[i][e] : db[i][e];
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        float v = cross[c];
#pragma unroll
        for (int q = 1; q < WARP_ROWS; ++q) v += cross[q * a.cols + c];
        out[slot + c] = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = col_of<VEC, WPR>(i);
        if (c < a.cols)
#pragma unroll
          for (int e = 0; e < VEC; ++e) out[slot + c + e] = k == 0 ? dw[i][e] : db[i][e];
      }
    }
  }
}

constexpr int RED_COLS = 32, RED_ROWS = 8;

// out[g][c] = sum over the group's parts of slots[g * parts + part][c]: RED_ROWS threads of a
// column take every RED_ROWS-th part, and their sums are added in order.  blockIdx.y: dw, db.
__global__ void __launch_bounds__(RED_COLS * RED_ROWS)
reduce_kernel(int64_t cols, int parts, const float* __restrict__ dw_slots, const float* __restrict__ db_slots,
              float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float s[RED_ROWS][RED_COLS];
  const int64_t blocks = (cols + RED_COLS - 1) / RED_COLS;
  const int64_t g = blockIdx.x / blocks;
  const int64_t c = (blockIdx.x - g * blocks) * RED_COLS + threadIdx.x % RED_COLS;
  const int y = threadIdx.x / RED_COLS;
  const float* in = blockIdx.y == 0 ? dw_slots : db_slots;
  float* out = blockIdx.y == 0 ? dw : db;
  pdl_wait();
  float v = 0.f;
  if (out && c < cols)
#pragma unroll 4
    for (int k = y; k < parts; k += RED_ROWS) v += in[(g * parts + k) * cols + c];
  s[y][threadIdx.x % RED_COLS] = v;
  __syncthreads();
  if (y == 0 && out && c < cols) {
#pragma unroll
    for (int k = 1; k < RED_ROWS; ++k) v += s[k][threadIdx.x];
    out[g * cols + c] = v;
  }
}

}  // namespace ln
}  // namespace la
