// clip.cuh -- global gradient norm over a list of tensors, and clipping (la_grad_norm,
// la_clip_grad_norm):  norm = sqrt(sum g^2),  out = g min(1, max_norm / (norm + 1e-6)).
//
// Bound by HBM: one read for the norm, one read and one write to clip (the norm is needed before
// the first write; a list that fits the L2 cache is read from HBM once).  1.87 GB: 1022 us, 5.5 TB/s over
// the three passes.  The list travels in the
// kernel's parameters, so a captured call needs no device table.  Tensors are cut into chunks; the
// blocks of a fixed grid take chunks in a fixed order and leave one fp64 sum each, and every block
// of the second kernel adds those sums in the same order.
#pragma once
#include "common.cuh"
#include "sm100.cuh"

namespace la {
namespace clip {

constexpr int THREADS = 256;
constexpr int CHUNK_BYTES = 32768;

// Up to CAP tensors.  chunk0[i] is the number of chunks before tensor i; flags: bit 0 = fp32.
template <int CAP>
struct Table {
  const void* in[CAP];
  void* out[CAP];
  int64_t numel[CAP];
  uint32_t chunk0[CAP];  // chunk0[i + 1] - chunk0[i] chunks; the list's total in `chunks`
  uint32_t chunks;
  int32_t count;
  uint32_t f32[(CAP + 31) / 32];
};

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) v += red[w];
  return v;
}

// Sum of squares of a few values, in fp32 where that neither overflows nor loses small values,
// else in fp64 (NaN and infinities come out right there).
template <int N>
__device__ __forceinline__ double squares(const float (&v)[N]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s += v[i] * v[i];
  // A square below 2^-126 (a subnormal, or 0) is off by 2^-150 at most: N of them are below
  // 2^-24 of a sum above 2^-120.
  if (s > 7.6e-37f && s < 3.0e38f) return double(s);
  double d = 0.0;
  if (s == 0.f) {  // all zero, as the gradients of unused embeddings are, or too small to square
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(v[i]));
    if (m == 0.f) return d;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) d += double(v[i]) * double(v[i]);
  return d;
}

__device__ __forceinline__ void unpack(const uint4& u, float (&v)[8]) {
  v[0] = bf16lo(u.x); v[1] = bf16hi(u.x); v[2] = bf16lo(u.y); v[3] = bf16hi(u.y);
  v[4] = bf16lo(u.z); v[5] = bf16hi(u.z); v[6] = bf16lo(u.w); v[7] = bf16hi(u.w);
}

// 16 bytes that are read once (per kernel): not worth a place in L1.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}

template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP>& t, uint32_t chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.chunk0[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The list's chunks in this block's order: calls f(tensor, first element, elements, is fp32).
template <int CAP, bool REVERSE, typename F>
__device__ __forceinline__ void for_chunks(const Table<CAP>& t, F&& f) {
  for (uint32_t i = blockIdx.x; i < t.chunks; i += gridDim.x) {
    const uint32_t c = REVERSE ? t.chunks - 1 - i : i;
    const int k = tensor_of(t, c);
    const bool is32 = (t.f32[k >> 5] >> (k & 31)) & 1u;
    const int64_t per = is32 ? CHUNK_BYTES / 4 : CHUNK_BYTES / 2;
    const int64_t e0 = int64_t(c - t.chunk0[k]) * per;
    const int64_t left = t.numel[k] - e0;
    f(k, e0, static_cast<int>(left < per ? left : per), is32);
  }
}

template <int CAP>
__global__ void __launch_bounds__(THREADS)
norm_kernel(const __grid_constant__ Table<CAP> t, double* __restrict__ partial) {
  __shared__ double red[THREADS / 32];
  pdl_trigger();
  double acc = 0.0;
  for_chunks<CAP, false>(t, [&](int k, int64_t e0, int n, bool is32) {
    const int tid = threadIdx.x;
    int done = 0;
    if (is32) {
      const float* p = static_cast<const float*>(t.in[k]) + e0;
      if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        const float4* p4 = reinterpret_cast<const float4*>(p);
        const int n4 = n >> 2;
#pragma unroll 4
        for (int i = tid; i < n4; i += THREADS) {
          const uint4 u = load16(p4 + i);
          const float v[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
          acc += squares(v);
        }
        done = n4 << 2;
      }
      for (int i = done + tid; i < n; i += THREADS) {
        const float v[1] = {p[i]};
        acc += squares(v);
      }
    } else {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(t.in[k]) + e0;
      if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        const uint4* p8 = reinterpret_cast<const uint4*>(p);
        const int n8 = n >> 3;
#pragma unroll 4
        for (int i = tid; i < n8; i += THREADS) {
          float v[8];
          unpack(load16(p8 + i), v);
          acc += squares(v);
        }
        done = n8 << 3;
      }
      for (int i = done + tid; i < n; i += THREADS) {
        const float v[1] = {__bfloat162float(p[i])};
        acc += squares(v);
      }
    }
  });
  acc = block_sum(acc, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

// The norm from the blocks' sums, the same value (and order of addition) in every thread.
__device__ __forceinline__ double total_norm(const double* partial, int parts, double* red) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += THREADS) v += partial[i];
  return sqrt(block_sum(v, red));
}

__global__ void __launch_bounds__(THREADS)
finish_kernel(const double* partial, int parts, float* __restrict__ norm) {
  __shared__ double red[THREADS / 32];
  pdl_wait();
  const double v = total_norm(partial, parts, red);
  if (threadIdx.x == 0) norm[0] = static_cast<float>(v);
}

// The chunks are taken last to first: the end of the list is what the norm kernel left in L2.  Reads
// past L1, stores that leave L2 first, 2 packs a thread at a time and 8 blocks an SM: 3.7 GB in 670 us
// (5.5 TB/s); with 4 blocks and 8 packs, or loads through L1, it took 870.
template <int CAP>
__global__ void __launch_bounds__(THREADS)
scale_kernel(const __grid_constant__ Table<CAP> t, const double* partial, int parts, float max_norm, float* norm) {
  __shared__ double red[THREADS / 32];
  pdl_trigger();
  pdl_wait();
  const double total = total_norm(partial, parts, red);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = static_cast<float>(total);
  const double ratio = double(max_norm) / (total + 1e-6);
  // A coefficient near fp32's smallest numbers would lose its bits: below 2^-100 it is taken 2^128 times as
  // large and 2^-64 is applied before it and after it (both exactly, or to results below fp32's range).
  const bool far = ratio < 0x1p-100;
  const float s = far ? 0x1p-64f : 1.f;
  const float c = ratio > 1.0 ? 1.f : static_cast<float>(far ? ratio * 0x1p128 : ratio);  // (NaN stays NaN)
  auto scaled = [&](float v) { return v * s * c * s; };
  for_chunks<CAP, true>(t, [&](int k, int64_t e0, int n, bool is32) {
    if (c == 1.f && t.in[k] == t.out[k]) return;  // nothing to change in place
    const int tid = threadIdx.x;
    int done = 0;
    if (is32) {
      const float* p = static_cast<const float*>(t.in[k]) + e0;
      float* o = static_cast<float*>(t.out[k]) + e0;
      if (((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(o)) & 15u) == 0) {
        const float4* p4 = reinterpret_cast<const float4*>(p);
        float4* o4 = reinterpret_cast<float4*>(o);
        const int n4 = n >> 2;
#pragma unroll 2
        for (int i = tid; i < n4; i += THREADS) {
          const uint4 u = load16(p4 + i);
          __stcs(o4 + i, make_float4(scaled(__uint_as_float(u.x)), scaled(__uint_as_float(u.y)),
                                     scaled(__uint_as_float(u.z)), scaled(__uint_as_float(u.w))));
        }
        done = n4 << 2;
      }
      for (int i = done + tid; i < n; i += THREADS) o[i] = scaled(p[i]);
    } else {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(t.in[k]) + e0;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(t.out[k]) + e0;
      if (((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(o)) & 15u) == 0) {
        const uint4* p8 = reinterpret_cast<const uint4*>(p);
        uint4* o8 = reinterpret_cast<uint4*>(o);
        const int n8 = n >> 3;
#pragma unroll 2
        for (int i = tid; i < n8; i += THREADS) {
          float v[8];
          unpack(load16(p8 + i), v);
          uint4 u;
          u.x = pack_bf16(scaled(v[0]), scaled(v[1]));
          u.y = pack_bf16(scaled(v[2]), scaled(v[3]));
          u.z = pack_bf16(scaled(v[4]), scaled(v[5]));
          u.w = pack_bf16(scaled(v[6]), scaled(v[7]));
          __stcs(o8 + i, u);
        }
        done = n8 << 3;
      }
      for (int i = done + tid; i < n; i += THREADS) o[i] = __float2bfloat16_rn(scaled(__bfloat162float(p[i])));
    }
  });
}

}  // namespace clip
}  // namespace la
