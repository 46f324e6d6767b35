// norm.cuh -- layer norm over the last dimension, forward and backward (la_layernorm_*).
//
//   y = (x - mean) rstd w_g + b_g;   with xh = (x - mean) rstd and a = dy w_g:
//   dx = rstd (a - mean(a) - xh mean(a xh)),  dw_g = sum dy xh,  db_g = sum dy.
//
// Both are bound by HBM: one read of x (and dy), one write of y (dx).  A row stays in registers
// between its read and its write, so the variance is the exact two-pass one.  75600 rows of 4096 in
// bf16: forward 238 us (5.2 TB/s), backward 349 (5.3); 32760 rows of 1000 in fp32: 45 us (5.8) and
// 69 (5.7).
//   Short rows (up to 512 channels; forward: up to a warp's 16 packs a lane) belong to a part of a
// warp, several rows at a time, without a barrier.  (Forward rows of 4096 in a block each took 300 to
// 385 us instead of 270.)
//   Longer rows belong to a block that walks its range of a group's rows, with the weight in
// registers; the rows to come are on their way to shared memory by bulk copies (a ring of up to 4
// rows), since loads into registers left too few bytes in flight (backward of two groups of 75600 rows:
// 1286 us, with the ring 707).
//   Rows that are not 16-byte aligned take the same kernels' one-element form (without the ring).
// In the backward pass a thread owns the same columns of every row it sees, so its shares of dw and
// db stay in registers until the block has walked its rows; blocks write them to their own slots,
// which a second kernel adds in order (no atomics: the same bits every time).
#pragma once
#include "common.cuh"
#include "sm100.cuh"

namespace la {
namespace ln {

// VEC elements of a row, as loaded: 16 bytes where rows are 16-byte aligned, else one element.  (bf16
// stays in words of two: as eight elements the compiler gives it eight registers.)
template <typename T, int VEC>
struct Pack {
  T v[VEC];
  __device__ __forceinline__ float get(int e) const { return static_cast<float>(v[e]); }
  __device__ __forceinline__ void set(const float (&f)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = T(f[e]);
  }
};
template <>
struct __align__(16) Pack<__nv_bfloat16, 8> {
  uint32_t v[4];
  __device__ __forceinline__ float get(int e) const { return (e & 1) ? bf16hi(v[e >> 1]) : bf16lo(v[e >> 1]); }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) v[e >> 1] = pack_bf16(f[e], f[e + 1]);
  }
};
template <>
struct __align__(16) Pack<float, 4> {
  float v[4];
  __device__ __forceinline__ float get(int e) const { return v[e]; }
  __device__ __forceinline__ void set(const float (&f)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = f[e];
  }
};

__device__ __forceinline__ void put(float& d, float x) { d = x; }
__device__ __forceinline__ void put(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

// A pack of a tensor that is read once: past the L1 cache, which the weights have.
template <typename P>
__device__ __forceinline__ P load_pack(const void* p) {
  if constexpr (sizeof(P) == 16) {
    uint4 u;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p) : "memory");
    return *reinterpret_cast<P*>(&u);
  } else {
    return *static_cast<const P*>(p);
  }
}
template <typename P>
__device__ __forceinline__ void store_pack(void* p, const P& v) {
  if constexpr (sizeof(P) == 16) {
    const uint4& u = *reinterpret_cast<const uint4*>(&v);
    *reinterpret_cast<uint4*>(p) = u;
  } else {
    *static_cast<P*>(p) = v;
  }
}

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

// Sum over the LPR lanes that share a row.
template <int LPR>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Args {
  int64_t rows, per_group, sx, sy, sdy, sdx;
  int32_t cols;
  float eps, inv_cols;
};

// ------------------------------------------------------------------------------- short rows
constexpr int WARPS = 4;  // of a block

// LPR lanes hold a row of NV packs each; a warp takes U * 32 / LPR rows at a time.
template <typename T, int VEC, int NV, int LPR, int U>
__global__ void __launch_bounds__(32 * WARPS)
forward_short(const Args a, const T* x, const float* __restrict__ weight, const float* __restrict__ bias, T* y,
              float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, li = lane % LPR;
  const int64_t row0 = (int64_t(blockIdx.x) * WARPS + (threadIdx.x >> 5)) * (U * RPW) + lane / LPR;
  Pack<T, VEC> p[U][NV];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LPR + li) * VEC;
      const int64_t row = row0 + u * RPW;
      if (c < a.cols && row < a.rows) p[u][i] = load_pack<Pack<T, VEC>>(x + row * a.sx + c);
    }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + u * RPW;
    const bool in = row < a.rows;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in && (i * LPR + li) * VEC < a.cols) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += p[u][i].get(e);
      }
    const float mu = lanes_sum<LPR>(s) * a.inv_cols;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in && (i * LPR + li) * VEC < a.cols) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float d = p[u][i].get(e) - mu;
          s += d * d;
        }
      }
    const float r = 1.f / sqrtf(lanes_sum<LPR>(s) * a.inv_cols + a.eps);
    if (!in) continue;
    if (mean && li == 0) {
      mean[row] = mu;
      rstd[row] = r;
    }
    const int64_t g = row / a.per_group * a.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LPR + li) * VEC;
      if (c >= a.cols) continue;
      float w[VEC], b[VEC];
      if (weight) load_w<VEC>(weight + g + c, w);
      if (bias) load_w<VEC>(bias + g + c, b);
      float t[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        t[e] = (p[u][i].get(e) - mu) * r;
        if (weight) t[e] *= w[e];
        if (bias) t[e] += b[e];
      }
      p[u][i].set(t);
      store_pack(y + row * a.sy + c, p[u][i]);
    }
  }
}

// Block `part` of group g takes every parts-th step of the group's rows and leaves its sums in slot
// g * parts + part of dw_out and db_out ([groups * parts][cols]).
template <typename T, int VEC, int NV, int LPR, int U>
__global__ void __launch_bounds__(32 * WARPS)
backward_short(const Args a, int parts, const T* x, const T* dy, const float* __restrict__ weight,
               const float* __restrict__ mean, const float* __restrict__ rstd, T* dx, float* dw_out, float* db_out) {
  constexpr int RPW = 32 / LPR, STEP = WARPS * U * RPW;
  extern __shared__ float cross[];  // [WARPS * RPW][cols]: the sums of the block's row slots, joined at the end
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, li = lane % LPR;
  const int64_t g = blockIdx.x / static_cast<uint32_t>(parts);
  const int part = static_cast<int>(blockIdx.x - g * parts);
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * LPR + li) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[i][e] = 1.f;
      dw[i][e] = db[i][e] = 0.f;
    }
    if (weight && c < a.cols) load_w<VEC>(weight + g * a.cols + c, w[i]);
  }
  for (int64_t j0 = int64_t(part) * STEP; j0 < a.per_group; j0 += int64_t(parts) * STEP) {
    Pack<T, VEC> px[U][NV], pd[U][NV];
    float mu[U], r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t j = j0 + (warp * U + u) * RPW + lane / LPR, row = g * a.per_group + j;
      const bool in = j < a.per_group;
      mu[u] = in ? mean[row] : 0.f;
      r[u] = in ? rstd[row] : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * LPR + li) * VEC;
        if (in && c < a.cols) {
          px[u][i] = load_pack<Pack<T, VEC>>(x + row * a.sx + c);
          pd[u][i] = load_pack<Pack<T, VEC>>(dy + row * a.sdy + c);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t j = j0 + (warp * U + u) * RPW + lane / LPR, row = g * a.per_group + j;
      const bool in = j < a.per_group;
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (in && (i * LPR + li) * VEC < a.cols) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float xh = (px[u][i].get(e) - mu[u]) * r[u], d = pd[u][i].get(e);
            dw[i][e] += d * xh;
            db[i][e] += d;
            s1 += d * w[i][e];
            s2 += d * w[i][e] * xh;
          }
        }
      const float c1 = lanes_sum<LPR>(s1) * a.inv_cols, c2 = lanes_sum<LPR>(s2) * a.inv_cols;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * LPR + li) * VEC;
        if (!in || c >= a.cols) continue;
        float t[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (px[u][i].get(e) - mu[u]) * r[u];
          t[e] = r[u] * (pd[u][i].get(e) * w[i][e] - c1 - xh * c2);
        }
        px[u][i].set(t);
        store_pack(dx + row * a.sdx + c, px[u][i]);
      }
    }
  }
  const int64_t slot = int64_t(blockIdx.x) * a.cols;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* out = k == 0 ? dw_out : db_out;
    if (!out) continue;
    // the block's row slots saw different rows of the same columns: join them in order
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LPR + li) * VEC;
      if (c < a.cols)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          cross[(warp * RPW + lane / LPR) * a.cols + c + e] = k == 0 ? dw[i][e] : db[i][e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += 32 * WARPS) {
      float v = cross[c];
#pragma unroll
      for (int q = 1; q < WARPS * RPW; ++q) v += cross[q * a.cols + c];
      out[slot + c] = v;
    }
  }
}

// ------------------------------------------------------------------------------- long rows
// A block of WPR warps per row.  RING: rows come through a ring of `stages` in shared memory (16-byte
// packs), else straight from global memory.
struct Ring {
  uint64_t full[4];
  int abort_flag;
};
// Thread 0 when a wait gave up: waits (with a limit) for the copies that it has issued, so that none
// lands in shared memory that is no longer the block's.
__device__ __forceinline__ void ring_drain(Ring& rg, int stages, uint32_t issued) {
  const uint32_t n = static_cast<uint32_t>(stages);
  for (uint32_t i = issued > n ? issued - n : 0; i < issued; ++i) mbar_wait_drain(&rg.full[i % n], (i / n) & 1);
}

// The sum of two values over the block's warps, in warp order; one barrier, and the next call's may
// follow at once (callers alternate the buffers).
template <int WPR>
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* red) {
  a = lanes_sum<32>(a);
  b = lanes_sum<32>(b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = make_float2(a, b);
  __syncthreads();
  const float2 t = lane < WPR ? red[lane] : make_float2(0.f, 0.f);
  return make_float2(lanes_sum<32>(t.x), lanes_sum<32>(t.y));
}

template <typename T, int VEC, int NV, int WPR, bool RING>
__global__ void __launch_bounds__(32 * WPR)
forward_long(const Args a, int parts, int stages, const T* x, const float* __restrict__ weight,
             const float* __restrict__ bias, T* y, float* __restrict__ mean, float* __restrict__ rstd) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float2 red[2][32];
  __shared__ Ring rg;
  const int64_t g = blockIdx.x / static_cast<uint32_t>(parts);
  const int part = static_cast<int>(blockIdx.x - g * parts);
  const uint32_t bytes = static_cast<uint32_t>(a.cols) * sizeof(T);
  const int64_t row0 = g * a.per_group;
  uint32_t issued = 0;  // (thread 0's)
  auto fetch = [&](int64_t j, int s) {
    if (j < a.per_group) {
      ++issued;
      mbar_arrive_expect_tx(&rg.full[s], bytes);
      if (!lose(LOSE_NORM_ROW)) bulk_load(ring + s * bytes, x + (row0 + j) * a.sx, bytes, &rg.full[s]);
    }
  };
  if (RING && threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&rg.full[s], 1);
    rg.abort_flag = 0;
    fence_mbar_init();
    for (int s = 0; s < stages; ++s) fetch(part + int64_t(s) * parts, s);
  }
  __syncthreads();
  float w[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * 32 * WPR + threadIdx.x) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[i][e] = 1.f;
      b[i][e] = 0.f;
    }
    if (weight && c < a.cols) load_w<VEC>(weight + g * a.cols + c, w[i]);
    if (bias && c < a.cols) load_w<VEC>(bias + g * a.cols + c, b[i]);
  }
  int s = 0;
  uint32_t ph = 0;
  for (int64_t j = part; j < a.per_group; j += parts) {
    const int64_t row = row0 + j;
    Pack<T, VEC> p[NV];
    if constexpr (RING) mbar_wait_near(&rg.full[s], ph, &rg.abort_flag);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * 32 * WPR + threadIdx.x) * VEC;
      if (c < a.cols)
        p[i] = RING ? *reinterpret_cast<const Pack<T, VEC>*>(ring + s * bytes + c * sizeof(T))
                    : load_pack<Pack<T, VEC>>(x + row * a.sx + c);
    }
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * 32 * WPR + int(threadIdx.x)) * VEC < a.cols) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v += p[i].get(e);
      }
    const float mu = block_sum2<WPR>(v, 0.f, red[0]).x * a.inv_cols;
    if constexpr (RING) {  // every thread has its part of the row: the stage can take another one
      if (*static_cast<volatile int*>(&rg.abort_flag)) break;
      if (threadIdx.x == 0) fetch(j + int64_t(stages) * parts, s);
      if (++s == stages) {
        s = 0;
        ph ^= 1;
      }
    }
    v = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * 32 * WPR + int(threadIdx.x)) * VEC < a.cols) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float d = p[i].get(e) - mu;
          v += d * d;
        }
      }
    const float r = 1.f / sqrtf(block_sum2<WPR>(v, 0.f, red[1]).x * a.inv_cols + a.eps);
    if (mean && threadIdx.x == 0) {
      mean[row] = mu;
      rstd[row] = r;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * 32 * WPR + threadIdx.x) * VEC;
      if (c >= a.cols) continue;
      float t[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        t[e] = (p[i].get(e) - mu) * r;
        if (weight) t[e] *= w[i][e];
        if (bias) t[e] += b[i][e];
      }
      p[i].set(t);
      store_pack(y + row * a.sy + c, p[i]);
    }
  }
  if (RING && threadIdx.x == 0 && rg.abort_flag) ring_drain(rg, stages, issued);
}

template <typename T, int VEC, int NV, int WPR, bool RING>
__global__ void __launch_bounds__(32 * WPR)
backward_long(const Args a, int parts, int stages, const T* x, const T* dy, const float* __restrict__ weight,
              const float* __restrict__ mean, const float* __restrict__ rstd, T* dx, float* dw_out, float* db_out) {
  extern __shared__ __align__(128) uint8_t ring[];  // stages of a row of x, then of dy
  __shared__ float2 red[2][32];
  __shared__ Ring rg;
  pdl_trigger();
  const int64_t g = blockIdx.x / static_cast<uint32_t>(parts);
  const int part = static_cast<int>(blockIdx.x - g * parts);
  const uint32_t bytes = static_cast<uint32_t>(a.cols) * sizeof(T);
  const int64_t row0 = g * a.per_group;
  uint32_t issued = 0;  // (thread 0's)
  auto fetch = [&](int64_t j, int s) {
    if (j < a.per_group) {
      ++issued;
      mbar_arrive_expect_tx(&rg.full[s], 2 * bytes);
      if (!lose(LOSE_NORM_ROW)) bulk_load(ring + (2 * s) * bytes, x + (row0 + j) * a.sx, bytes, &rg.full[s]);
      bulk_load(ring + (2 * s + 1) * bytes, dy + (row0 + j) * a.sdy, bytes, &rg.full[s]);
    }
  };
  if (RING && threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&rg.full[s], 1);
    rg.abort_flag = 0;
    fence_mbar_init();
    for (int s = 0; s < stages; ++s) fetch(part + int64_t(s) * parts, s);
  }
  __syncthreads();
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * 32 * WPR + threadIdx.x) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[i][e] = 1.f;
      dw[i][e] = db[i][e] = 0.f;
    }
    if (weight && c < a.cols) load_w<VEC>(weight + g * a.cols + c, w[i]);
  }
  int s = 0, buf = 0;
  uint32_t ph = 0;
  float mu = 0.f, r = 0.f;
  if (part < a.per_group) {
    mu = mean[row0 + part];
    r = rstd[row0 + part];
  }
  for (int64_t j = part; j < a.per_group; j += parts) {
    const int64_t row = row0 + j;
    Pack<T, VEC> px[NV], pd[NV];
    if constexpr (RING) mbar_wait_near(&rg.full[s], ph, &rg.abort_flag);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * 32 * WPR + threadIdx.x) * VEC;
      if (c < a.cols) {
        px[i] = RING ? *reinterpret_cast<const Pack<T, VEC>*>(ring + (2 * s) * bytes + c * sizeof(T))
                     : load_pack<Pack<T, VEC>>(x + row * a.sx + c);
        pd[i] = RING ? *reinterpret_cast<const Pack<T, VEC>*>(ring + (2 * s + 1) * bytes + c * sizeof(T))
                     : load_pack<Pack<T, VEC>>(dy + row * a.sdy + c);
      }
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * 32 * WPR + int(threadIdx.x)) * VEC < a.cols) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (px[i].get(e) - mu) * r, d = pd[i].get(e);
          dw[i][e] += d * xh;
          db[i][e] += d;
          s1 += d * w[i][e];
          s2 += d * w[i][e] * xh;
        }
      }
    const float2 c12 = block_sum2<WPR>(s1, s2, red[buf]);
    buf ^= 1;
    const float mu0 = mu, r0 = r;
    if (j + parts < a.per_group) {  // the next row's
      mu = mean[row + parts];
      r = rstd[row + parts];
    }
    if constexpr (RING) {
      if (*static_cast<volatile int*>(&rg.abort_flag)) break;
      if (threadIdx.x == 0) fetch(j + int64_t(stages) * parts, s);
      if (++s == stages) {
        s = 0;
        ph ^= 1;
      }
    }
    const float c1 = c12.x * a.inv_cols, c2 = c12.y * a.inv_cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * 32 * WPR + threadIdx.x) * VEC;
      if (c >= a.cols) continue;
      float t[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (px[i].get(e) - mu0) * r0;
        t[e] = r0 * (pd[i].get(e) * w[i][e] - c1 - xh * c2);
      }
      px[i].set(t);
      store_pack(dx + row * a.sdx + c, px[i]);
    }
  }
  if (RING && threadIdx.x == 0 && rg.abort_flag) ring_drain(rg, stages, issued);
  const int64_t slot = int64_t(blockIdx.x) * a.cols;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * 32 * WPR + threadIdx.x) * VEC;
    if (c >= a.cols) continue;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (dw_out) dw_out[slot + c + e] = dw[i][e];
      if (db_out) db_out[slot + c + e] = db[i][e];
    }
  }
}

constexpr int RED_COLS = 32, RED_ROWS = 32;

// out[g][c] = sum over the group's parts of slots[g * parts + part][c]: RED_ROWS threads of a
// column take every RED_ROWS-th part, and their sums are added in order.  blockIdx.y: dw, db.  (With 8
// threads a column it took 20 of the 76 us of 32760 rows of 1000; with 32 the whole takes 69.)
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
#pragma unroll 8
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
