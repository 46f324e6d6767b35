// block_api.cu -- the part of the C ABI (include/la.h) for the operators of the block around the
// token mixer: cross attention, layer norm, gradient norm and clipping.  Argument checks, work
// planning and kernel launches.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <utility>

#include <cuda.h>
#include <cuda_runtime.h>

#include "la.h"
#include "host.cuh"
#include "common.cuh"
#include "sm100.cuh"
#include "norm.cuh"
#include "clip.cuh"
#include "cross_simt.cuh"
#include "cross_few.cuh"
#include "cross_tc.cuh"
#include "cross_bwd_tc.cuh"

namespace la {
cudaError_t take_block_error(unsigned int* value) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_la_error, sizeof *value);
  if (e != cudaSuccess || *value == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_la_error, &zero, sizeof zero);
}
}  // namespace la

namespace {

la::KernelTable g_kernels;

template <typename F>
int set_smem(F* kern, size_t bytes) { return g_kernels.smem(kern, bytes); }
template <typename F>
bool launch_regs(F* kern, uint32_t regs) { return g_kernels.regs(kern, regs); }

using la::align256;
using la::aligned16;
using la::current_sm_count;
using la::g_last_launches;
using la::launch_k;

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 1024;

size_t elem_size(int32_t dtype) { return dtype == LA_BF16 ? 2 : 4; }

// ------------------------------------------------------------------------------- cross attention
enum Tensor { TQ, TK, TV, TO, TDO, TDQ, TDK, TDV, TENSORS };

struct View {
  int64_t heads, tokens;
  la_strides s;
  bool output;
};

void cross_views(const la_cross_problem& p, View (&v)[TENSORS]) {
  v[TQ] = {p.H, p.Nq, p.q, false};
  v[TK] = {p.Hkv, p.Nk, p.k, false};
  v[TV] = {p.Hkv, p.Nk, p.v, false};
  v[TO] = {p.H, p.Nq, p.o, true};
  v[TDO] = {p.H, p.Nq, p.dout, false};
  v[TDQ] = {p.H, p.Nq, p.dq, true};
  v[TDK] = {p.Hkv, p.Nk, p.dk, true};
  v[TDV] = {p.Hkv, p.Nk, p.dv, true};
}

// The strides of a tensor that has elements: positive multiples of 16 bytes where the extent is
// above 1, offsets within 2^62 bytes, and no overlap within an output.
int check_strides(const la_cross_problem& p, const View& v) {
  const int64_t ext[3] = {p.B, v.heads, v.tokens};
  const int64_t str[3] = {v.s.b, v.s.h, v.s.n};
  if (ext[0] == 0 || ext[1] == 0 || ext[2] == 0) return LA_OK;
  const int64_t per16 = 16 / int64_t(elem_size(p.dtype));
  std::pair<int64_t, int64_t> dim[3];
  int n = 0;
  for (int i = 0; i < 3; ++i) {
    if (ext[i] == 1) continue;
    if (str[i] <= 0) return LA_ERR_SHAPE;
    if (str[i] % per16) return LA_ERR_ALIGN;
    if (double(str[i]) * double(ext[i]) > 1.0e18) return LA_ERR_SHAPE;
    dim[n++] = {str[i], ext[i]};
  }
  if (!v.output) return LA_OK;
  std::sort(dim, dim + n);
  int64_t span = p.d;  // elements from the first to one past the last of the dimensions so far
  for (int i = 0; i < n; ++i) {
    if (dim[i].first < span) return LA_ERR_SHAPE;
    span += dim[i].first * (dim[i].second - 1);
  }
  return LA_OK;
}

int validate(const la_cross_problem* p, bool backward) {
  if (!p) return LA_ERR_NULL;
  if (p->B < 0 || p->H < 0 || p->Hkv < 0 || p->Nq < 0 || p->Nk < 0) return LA_ERR_SHAPE;
  if (p->dtype != LA_BF16 && p->dtype != LA_F32) return LA_ERR_UNSUPPORTED;
  if (p->flags & ~uint32_t(LA_FLAG_FORCE_SIMT)) return LA_ERR_UNSUPPORTED;
  if (p->d != 32 && p->d != 64 && p->d != 128) return LA_ERR_UNSUPPORTED;
  if (!(p->scale > 0.f) || !std::isfinite(p->scale)) return LA_ERR_SHAPE;
  const int64_t lim = int64_t(1) << 31;
  if (p->B >= lim || p->H >= lim || p->Nq > kMaxTokens || p->Nk > kMaxTokens) return LA_ERR_SHAPE;
  if (p->H > 0 && (p->Hkv == 0 || p->H % p->Hkv)) return LA_ERR_SHAPE;
  if (p->H == 0 && p->Hkv != 0) return LA_ERR_SHAPE;
  // tiles and rows stay in 32 (grids) and 62 (offsets) bits
  const double bh = double(p->B) * double(p->H);
  if (bh * (double(p->Nq) / 64 + 1) >= double(lim) / 64 || bh * (double(p->Nk) / 64 + 1) >= double(lim) / 64)
    return LA_ERR_SHAPE;
  View v[TENSORS];
  cross_views(*p, v);
  for (int i = 0; i < (backward ? TENSORS : TDO); ++i)
    if (const int rc = check_strides(*p, v[i])) return rc;
  return LA_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a long axis is split over blocks, whose parts are joined afterwards: the fewest parts that
// (nearly) bring the last wave of blocks (`slots` at a time) to an end with the others.  A part has
// `least` tiles or more and costs `extra` of its own (as it starts, and its sums' way through memory).
// Parts for every SM whatever the waves are slower: forward of 32 heads 1024 x 1024, 66 instead of
// 27 us; 20 heads 1000 x 2000 (d = 64), 62 instead of 39; 100 heads 256 x 8192, 184 instead of 153.
struct Split {
  int parts, per;  // parts * per >= tiles
};
Split split_waves(int64_t tiles, int64_t blocks, int64_t slots, int64_t least, int64_t extra) {
  Split best = {1, static_cast<int>(std::max<int64_t>(tiles, 1))};
  if (tiles <= 0 || blocks <= 0) return best;
  const int64_t most = std::min<int64_t>(ceil_div(tiles, least), la::xs::MAX_SPLITS);
  double cost = double(ceil_div(blocks, slots)) * double(tiles + extra);
  for (int64_t w = 1; w <= 8; ++w) {  // the most parts that take w waves
    const int64_t s = std::min(w * slots / blocks, most);
    if (s < 2) continue;
    const int64_t per = ceil_div(tiles, s), parts = ceil_div(tiles, per);
    const double c = double(ceil_div(blocks * parts, slots)) * double(per + extra);
    if (c < 0.97 * cost) {
      cost = c;
      best = {static_cast<int>(parts), static_cast<int>(per)};
    }
  }
  return best;
}

constexpr int64_t kLongMask = 32768;

struct CrossPlan {
  bool tc;                       // tensor-core kernels (bf16)
  bool few;                      // forward: few rows per key head
  int64_t rows, keys;            // B * H * Nq, B * Hkv * Nk
  int64_t q_tiles, k_tiles;      // per head
  int64_t pairs;                 // pairs of 128-query tiles per head (tensor cores)
  int64_t pad;                   // rows per head of the gathered keys
  Split fwd, dq, dkv;
  size_t off_kc, off_vc, off_count, off_place, off_spans;  // gathered keys
  size_t off_o, off_ml;          // forward: partial outputs, maxima and sums
  size_t off_delta, off_part;    // gradients: D_i, partial sums (dQ, then dK and dV)
  size_t total;
};

// `uses`: la_cross_use, of which LA_CROSS_FORWARD or LA_CROSS_BACKWARD says whose workspace it is.
CrossPlan cross_plan(const la_cross_problem& p, int sm, unsigned uses) {
  CrossPlan c;
  std::memset(&c, 0, sizeof c);
  c.rows = p.B * p.H * p.Nq;
  c.keys = p.B * p.Hkv * p.Nk;
  c.q_tiles = ceil_div(p.Nq, la::xs::BT);
  c.k_tiles = ceil_div(p.Nk, la::xs::BT);
  const int64_t group = p.Hkv > 0 ? p.H / p.Hkv : 1;
  c.tc = p.dtype == LA_BF16 && !(p.flags & LA_FLAG_FORCE_SIMT) && c.rows > 0 && c.keys > 0;
  c.pairs = ceil_div(p.Nq, 2 * la::xt::BM);
  c.pad = ceil_div(p.Nk, 16) * 16;
  // A key head's rows in one block: one pass over the keys for all of them, where tiles of 64 or 128
  // rows would be all but empty and read them once for every query head.  16384 keys, 8 x 8 key heads:
  // 1 row 88 us (tensor cores: 137), 8 query heads of 1 row 175 (896); a single query head of 8 rows
  // takes 175 here and 137 there, so that from 5 rows on it goes there.
  const int64_t most = c.tc && group == 1 ? la::xf::MAX_ROWS / 2 : la::xf::MAX_ROWS;
  c.few = !(p.flags & LA_FLAG_FORCE_SIMT) && c.rows > 0 && c.keys > 0 && group * p.Nq <= most;
  // (Two blocks of up to 4 rows share an SM, and the keys are split into whole waves of them: 9 parts
  // take 100 us, 4 or 13 parts 105 and 18 parts 110, for 4 rows of the above.)
  c.fwd = c.few ? split_waves(c.k_tiles, p.B * p.Hkv, (group * p.Nq <= 4 ? 2 : 1) * int64_t(sm), 4, 2)
          : c.tc ? split_waves(ceil_div(p.Nk, la::xt::BN), p.B * p.H * c.pairs, sm, 4, 4)
               : split_waves(c.k_tiles, p.B * p.H * c.q_tiles, 2 * int64_t(sm), 2, 1);
  const int64_t q128 = ceil_div(p.Nq, la::xt::BM), k128 = ceil_div(p.Nk, la::xt::BN);
  // CUDA cores: whole waves too (as many parts as bring two blocks to every SM took 760 instead of 625 us
  // for 32 heads of 4000 queries and 300 keys, d = 32).  The gradients' blocks of d = 128 fill an SM.
  const int64_t slots = p.d == 128 ? sm : 2 * int64_t(sm);
  c.dq = c.tc ? split_waves(k128, p.B * p.H * q128, sm, 4, 4) : split_waves(c.k_tiles, p.B * p.H * c.q_tiles, slots, 2, 1);
  c.dkv = c.tc ? split_waves(q128 * group, p.B * p.Hkv * k128, sm, 4, 3)
               : split_waves(c.q_tiles * group, p.B * p.Hkv * c.k_tiles, slots, 2, 1);
  const size_t D = size_t(p.d);
  const bool back = (uses & LA_CROSS_BACKWARD) != 0;
  size_t off = 0;
  // (a few rows read K and V where they are; lengths alone end the CUDA-core kernels' walk)
  if (c.keys > 0 && (back || !c.few) && (uses & (c.tc ? LA_CROSS_LENGTHS | LA_CROSS_MASK : LA_CROSS_MASK))) {
    const size_t rows = size_t(p.B) * size_t(p.Hkv) * size_t(c.pad) * D * elem_size(p.dtype);
    c.off_kc = 0;
    c.off_vc = align256(rows);
    c.off_count = align256(c.off_vc + rows);
    c.off_place = align256(c.off_count + size_t(p.B) * 4);
    c.off_spans = align256(c.off_place + size_t(p.B) * size_t(p.Nk) * 4);
    off = align256(c.off_spans + size_t(p.B) * size_t(ceil_div(p.Nk, la::xs::G_SPAN)) * 4);
  }
  if (back) {
    c.off_delta = off;
    c.off_part = align256(c.off_delta + size_t(c.rows) * 4);
    const size_t part_dq = c.dq.parts > 1 ? size_t(c.dq.parts) * size_t(c.rows) * D * 4 : 0;
    const size_t part_kv = c.keys > 0 ? 2 * size_t(c.dkv.parts) * size_t(c.keys) * D * 4 : 0;
    c.total = align256(c.off_part + std::max(part_dq, part_kv));
  } else {
    c.total = off;
    if (c.fwd.parts > 1) {
      c.off_o = off;
      c.off_ml = align256(c.off_o + size_t(c.fwd.parts) * size_t(c.rows) * D * 4);
      c.total = align256(c.off_ml + size_t(c.fwd.parts) * size_t(c.rows) * 8);
    }
  }
  return c;
}

// What a call with these optional tensors uses.
unsigned uses_of(unsigned call, const int32_t* kv_len, const uint8_t* mask) {
  return call | (kv_len ? LA_CROSS_LENGTHS : 0) | (mask ? LA_CROSS_MASK : 0);
}

la::xs::Str str(const la_strides& s) { return {s.b, s.h, s.n}; }

la::xs::Args cross_args(const la_cross_problem& p, const CrossPlan& c, const int32_t* kv_len, const uint8_t* mask) {
  la::xs::Args a;
  std::memset(&a, 0, sizeof a);
  a.B = p.B; a.H = p.H; a.Hkv = p.Hkv; a.Nq = p.Nq; a.Nk = p.Nk;
  a.q_tiles = c.q_tiles;
  a.k_tiles = c.k_tiles;
  a.rows = c.rows;
  a.group = static_cast<int32_t>(p.Hkv > 0 ? p.H / p.Hkv : 1);
  a.scale = p.scale;
  a.q = str(p.q); a.k = str(p.k); a.v = str(p.v); a.o = str(p.o);
  a.dout = str(p.dout); a.dq = str(p.dq); a.dk = str(p.dk); a.dv = str(p.dv);
  a.kv_len = kv_len;
  a.mask = mask;
  return a;
}

void use(la::xs::Args& a, const Split& s) {
  a.splits = s.parts;
  a.tiles_per_split = s.per;
}

// Gathers the attended keys into the workspace (see gather_kernel).
template <int D, typename T>
int gather_keys(const la_cross_problem& p, const CrossPlan& c, const la::xs::Args& a, const void* K, const void* V, uint8_t* ws,
                cudaStream_t st, int* nl) {
  const int64_t grid = ceil_div(p.Nk, la::xs::G_KEYS) * p.Hkv * p.B;
  // A block counts the mask before its keys; of long masks, from sums of spans, which a kernel more
  // takes (whole forward calls with and without them: 8192 keys 22.7 and 21.7 us, 32768: 43.2 and 45.2,
  // 262144: 235 and 318).
  int32_t* spans = nullptr;
  if (a.mask && p.Nk >= kLongMask) {
    spans = reinterpret_cast<int32_t*>(ws + c.off_spans);
    if (launch_k(la::xs::count_kernel, dim3(unsigned(ceil_div(p.Nk, la::xs::G_SPAN) * p.B)), la::xs::G_THREADS, 0, st, false,
                 p.Nk, a.kv_len, a.mask, spans))
      return LA_ERR_CUDA;
    ++*nl;
  }
  if (launch_k(la::xs::gather_kernel<T, D / (16 / int(sizeof(T)))>, dim3(unsigned(grid)), la::xs::G_THREADS, 0, st, spans != nullptr, p.Hkv,
               p.Nk, c.pad, static_cast<const T*>(K), static_cast<const T*>(V), a.k, a.v, a.kv_len, a.mask, spans,
               reinterpret_cast<T*>(ws + c.off_kc), reinterpret_cast<T*>(ws + c.off_vc),
               reinterpret_cast<int32_t*>(ws + c.off_count), reinterpret_cast<int32_t*>(ws + c.off_place)))
    return LA_ERR_CUDA;
  ++*nl;
  return LA_OK;
}
la::xs::Str gathered(const la_cross_problem& p, const CrossPlan& c) { return {p.Hkv * c.pad * p.d, c.pad * p.d, p.d}; }

// With a mask, the CUDA-core kernels walk the gathered keys: what is left out costs nothing then, and
// a mask's holes are spread over all tiles.  (Lengths alone end the walk.)
template <int D, typename T>
int gather_masked(const la_cross_problem& p, const CrossPlan& c, la::xs::Args* a, const void** K, const void** V, uint8_t* ws,
                  cudaStream_t st, int* nl) {
  if (!a->mask || c.keys == 0) return LA_OK;
  if (const int rc = gather_keys<D, T>(p, c, *a, *K, *V, ws, st, nl)) return rc;
  *K = ws + c.off_kc;
  *V = ws + c.off_vc;
  a->k = a->v = gathered(p, c);
  a->kv_len = reinterpret_cast<const int32_t*>(ws + c.off_count);
  a->mask = nullptr;
  return LA_OK;
}

template <int D, typename T>
int cross_forward_simt(const la_cross_problem& p, const CrossPlan& c, la::xs::Args a, const void* Q, const void* K,
                       const void* V, void* O, float* lse, uint8_t* ws, cudaStream_t st, int* nl) {
  const int before = *nl;
  if (const int rc = gather_masked<D, T>(p, c, &a, &K, &V, ws, st, nl)) return rc;
  use(a, c.fwd);
  float* part_o = reinterpret_cast<float*>(ws + c.off_o);
  float2* part_ml = reinterpret_cast<float2*>(ws + c.off_ml);
  const size_t smem = la::xs::fwd_smem<D>();
  if (set_smem(la::xs::forward_kernel<D, T>, smem)) return LA_ERR_CUDA;
  if (launch_k(la::xs::forward_kernel<D, T>, dim3(unsigned(c.q_tiles * c.fwd.parts * p.B * p.H)), la::xs::THREADS, smem, st,
               *nl > before, a, static_cast<const T*>(Q), static_cast<const T*>(K), static_cast<const T*>(V),
               static_cast<T*>(O), lse, part_o, part_ml))
    return LA_ERR_CUDA;
  ++*nl;
  if (c.fwd.parts > 1) {
    if (launch_k(la::xs::join_kernel<D, T>, dim3(unsigned(c.rows)), 32 * la::xs::JOIN_WARPS, 0, st, true, a, part_o, part_ml, static_cast<T*>(O), lse))
      return LA_ERR_CUDA;
    ++*nl;
  }
  return LA_OK;
}

template <int D, typename T>
int cross_backward_simt(const la_cross_problem& p, const CrossPlan& c, la::xs::Args a, const void* Q, const void* K,
                        const void* V, const void* O, const float* lse, const void* dO, void* dQ, void* dK, void* dV,
                        uint8_t* ws, cudaStream_t st, int* nl) {
  float* delta = reinterpret_cast<float*>(ws + c.off_delta);
  float* part = reinterpret_cast<float*>(ws + c.off_part);
  const size_t smem = la::xs::bwd_smem<D>();
  const bool masked = a.mask != nullptr && c.keys > 0;
  if (const int rc = gather_masked<D, T>(p, c, &a, &K, &V, ws, st, nl)) return rc;
  const T *q = static_cast<const T*>(Q), *k = static_cast<const T*>(K), *v = static_cast<const T*>(V),
          *g = static_cast<const T*>(dO);
  bool pdl = masked;
  if (c.rows > 0) {
    if (launch_k(la::xs::delta_kernel<D, T>, dim3(unsigned(p.B * p.H * ceil_div(p.Nq, la::xs::delta_rows<D, T>()))), la::xs::THREADS, 0, st,
                 pdl, a, static_cast<const T*>(O), g, delta))
      return LA_ERR_CUDA;
    use(a, c.dq);
    if (set_smem(la::xs::dq_kernel<D, T>, smem)) return LA_ERR_CUDA;
    if (launch_k(la::xs::dq_kernel<D, T>, dim3(unsigned(c.q_tiles * c.dq.parts * p.B * p.H)), la::xs::THREADS, smem, st, true,
                 a, q, k, v, g, lse, delta, static_cast<T*>(dQ), part))
      return LA_ERR_CUDA;
    *nl += 2;
    if (c.dq.parts > 1) {
      if (launch_k(la::xs::sum_rows_kernel<D, T>, dim3(unsigned(ceil_div(c.rows * (D / 2), la::xs::THREADS))), la::xs::THREADS, 0,
                   st, true, a, part, static_cast<T*>(dQ)))
        return LA_ERR_CUDA;
      ++*nl;
    }
    pdl = true;
  }
  if (c.keys > 0) {
    use(a, c.dkv);
    const bool parts = c.dkv.parts > 1 || masked;
    float* part_k = parts ? part : nullptr;
    float* part_v = part + int64_t(c.dkv.parts) * c.keys * D;
    if (set_smem(la::xs::dkv_kernel<D, T>, smem)) return LA_ERR_CUDA;
    if (launch_k(la::xs::dkv_kernel<D, T>, dim3(unsigned(c.k_tiles * c.dkv.parts * p.B * p.Hkv)), la::xs::THREADS, smem, st, pdl,
                 a, q, k, v, g, lse, delta, static_cast<T*>(dK), static_cast<T*>(dV), part_k, part_v))
      return LA_ERR_CUDA;
    ++*nl;
    if (parts) {
      if (launch_k(la::xs::sum_keys_kernel<D, T>, dim3(unsigned(ceil_div(c.keys * (D / 2), la::xs::THREADS)), 2), la::xs::THREADS,
                   0, st, true, c.keys, p.Hkv, p.Nk, c.dkv.parts, part, part_v,
                   masked ? reinterpret_cast<const int32_t*>(ws + c.off_place) : static_cast<const int32_t*>(nullptr),
                   static_cast<T*>(dK), static_cast<T*>(dV), a.dk, a.dv))
        return LA_ERR_CUDA;
      ++*nl;
    }
  }
  return LA_OK;
}

// A [B, heads, tokens, d] bf16 view as a 4D tensor {d, tokens, heads, B}; boxes of 64 channels x 128
// tokens, 128-byte swizzle (the canonical UMMA operand layout).  Channels and tokens outside read 0.
bool make_tmap4(CUtensorMap* m, const void* base, int64_t d, int64_t tokens, int64_t heads, int64_t B, const la::xs::Str& s) {
  cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(tokens), cuuint64_t(heads), cuuint64_t(B)};
  // (the stride of a dimension of extent 1 is never used: any legal value)
  cuuint64_t strides[3] = {tokens > 1 ? cuuint64_t(s.n) * 2 : 256, heads > 1 ? cuuint64_t(s.h) * 2 : 256,
                           B > 1 ? cuuint64_t(s.b) * 2 : 256};
  for (cuuint64_t x : strides)
    if (x >= cuuint64_t(1) << 40) return false;
  cuuint32_t box[4] = {64, 128, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return la::encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// The keys as the tensor-core kernels read them: the tensors themselves, or (with lengths or a
// mask) the attended rows, gathered.
struct Keys {
  CUtensorMap k, v;
  const int32_t* count;
};

template <int D>
int prepare_keys(const la_cross_problem& p, const CrossPlan& c, const la::xs::Args& a, const void* K, const void* V,
                 uint8_t* ws, cudaStream_t st, Keys* out, int* nl) {
  out->count = nullptr;
  if (!a.kv_len && !a.mask)
    return make_tmap4(&out->k, K, D, p.Nk, p.Hkv, p.B, a.k) && make_tmap4(&out->v, V, D, p.Nk, p.Hkv, p.B, a.v) ? LA_OK
                                                                                                          : LA_ERR_CUDA;
  const la::xs::Str s = gathered(p, c);
  if (!make_tmap4(&out->k, ws + c.off_kc, D, c.pad, p.Hkv, p.B, s) || !make_tmap4(&out->v, ws + c.off_vc, D, c.pad, p.Hkv, p.B, s))
    return LA_ERR_CUDA;
  out->count = reinterpret_cast<const int32_t*>(ws + c.off_count);
  return gather_keys<D, __nv_bfloat16>(p, c, a, K, V, ws, st, nl);
}

template <int D>
int cross_forward_tc(const la_cross_problem& p, const CrossPlan& c, la::xs::Args a, const void* Q, const void* K,
                     const void* V, void* O, float* lse, uint8_t* ws, int sm, cudaStream_t st, int* nl) {
  constexpr int DP = D < 64 ? 64 : D;
  CUtensorMap tq;
  Keys keys;
  if (!make_tmap4(&tq, Q, D, p.Nq, p.H, p.B, a.q)) return LA_ERR_CUDA;
  if (const int rc = prepare_keys<D>(p, c, a, K, V, ws, st, &keys, nl)) return rc;
  la::xt::Args t;
  std::memset(&t, 0, sizeof t);
  t.B = p.B; t.H = p.H; t.Nq = p.Nq; t.Nk = p.Nk;
  t.rows = c.rows;
  t.pairs = static_cast<int32_t>(c.pairs);
  t.group = a.group;
  t.splits = c.fwd.parts;
  t.per = c.fwd.per;
  t.total = p.B * p.H * c.pairs * c.fwd.parts;
  t.fd_pairs = la::make_fastdiv(uint32_t(t.pairs));
  t.fd_splits = la::make_fastdiv(uint32_t(t.splits));
  t.fd_H = la::make_fastdiv(uint32_t(p.H));
  t.c = p.scale * la::xt::LOG2E;
  t.count = keys.count;
  t.o = a.o;
  // 32-byte stores where every row of O starts on a 32-byte boundary
  const bool wide = (reinterpret_cast<uintptr_t>(O) & 31) == 0 && (p.Nq == 1 || p.o.n % 16 == 0) &&
                    (p.H == 1 || p.o.h % 16 == 0) && (p.B == 1 || p.o.b % 16 == 0);
  auto kern = la::xt::forward_kernel<DP, D>;
  const size_t smem = la::xt::Cfg<DP>::SMEM;
  if (set_smem(kern, smem) || !launch_regs(kern, la::xt::REGS_LAUNCH)) return LA_ERR_CUDA;
  float* part_o = reinterpret_cast<float*>(ws + c.off_o);
  float2* part_ml = reinterpret_cast<float2*>(ws + c.off_ml);
  if (launch_k(kern, dim3(unsigned(std::min<int64_t>(t.total, sm))), la::xt::THREADS, smem, st, keys.count != nullptr, tq,
               keys.k, keys.v, t, static_cast<__nv_bfloat16*>(O), lse, part_o, part_ml, int(wide)))
    return LA_ERR_CUDA;
  ++*nl;
  if (c.fwd.parts > 1) {
    use(a, c.fwd);
    if (launch_k(la::xs::join_kernel<D, __nv_bfloat16>, dim3(unsigned(c.rows)), 32 * la::xs::JOIN_WARPS, 0, st, true, a, part_o, part_ml, static_cast<__nv_bfloat16*>(O), lse))
      return LA_ERR_CUDA;
    ++*nl;
  }
  return LA_OK;
}

template <int D>
int cross_backward_tc(const la_cross_problem& p, const CrossPlan& c, la::xs::Args a, const void* Q, const void* K,
                      const void* V, const void* O, const float* lse, const void* dO, void* dQ, void* dK, void* dV,
                      uint8_t* ws, int sm, cudaStream_t st, int* nl) {
  constexpr int DP = D < 64 ? 64 : D;
  using T = __nv_bfloat16;
  CUtensorMap tq, tg;
  Keys keys;
  if (!make_tmap4(&tq, Q, D, p.Nq, p.H, p.B, a.q) || !make_tmap4(&tg, dO, D, p.Nq, p.H, p.B, a.dout)) return LA_ERR_CUDA;
  if (const int rc = prepare_keys<D>(p, c, a, K, V, ws, st, &keys, nl)) return rc;
  float* delta = reinterpret_cast<float*>(ws + c.off_delta);
  float* part = reinterpret_cast<float*>(ws + c.off_part);
  la::xb::Args t;
  std::memset(&t, 0, sizeof t);
  t.B = p.B; t.H = p.H; t.Hkv = p.Hkv; t.Nq = p.Nq; t.Nk = p.Nk;
  t.rows = c.rows;
  t.keys = c.keys;
  t.q_tiles = static_cast<int32_t>(ceil_div(p.Nq, la::xt::BM));
  t.group = a.group;
  t.c = p.scale * la::xt::LOG2E;
  t.scale = p.scale;
  t.count = keys.count;
  t.dq = a.dq;
  const bool wide = (reinterpret_cast<uintptr_t>(dQ) & 31) == 0 && (p.Nq == 1 || p.dq.n % 16 == 0) &&
                    (p.H == 1 || p.dq.h % 16 == 0) && (p.B == 1 || p.dq.b % 16 == 0);
  auto kq = la::xb::dq_kernel<DP, D>;
  auto kk = la::xb::dkv_kernel<DP, D>;
  const size_t mq = la::xb::CfgQ<DP>::SMEM, mk = la::xb::CfgK<DP>::SMEM;
  if (set_smem(kq, mq) || set_smem(kk, mk) || !launch_regs(kq, la::xb::REGS_LAUNCH) || !launch_regs(kk, la::xb::REGS_LAUNCH))
    return LA_ERR_CUDA;
  if (launch_k(la::xs::delta_kernel<D, T>, dim3(unsigned(p.B * p.H * ceil_div(p.Nq, la::xs::delta_rows<D, T>()))), la::xs::THREADS, 0, st,
               keys.count != nullptr, a, static_cast<const T*>(O), static_cast<const T*>(dO), delta))
    return LA_ERR_CUDA;
  ++*nl;
  t.tiles = t.q_tiles;
  t.splits = c.dq.parts;
  t.per = c.dq.per;
  t.total = p.B * p.H * int64_t(t.tiles) * t.splits;
  auto divisions = [&](int64_t heads) {
    t.fd_tiles = la::make_fastdiv(uint32_t(t.tiles));
    t.fd_splits = la::make_fastdiv(uint32_t(t.splits));
    t.fd_heads = la::make_fastdiv(uint32_t(heads));
  };
  divisions(p.H);
  if (launch_k(kq, dim3(unsigned(std::min<int64_t>(t.total, sm))), la::xb::THREADS, mq, st, true, tq, tg, keys.k, keys.v, t,
               lse, delta, static_cast<T*>(dQ), part, int(wide)))
    return LA_ERR_CUDA;
  ++*nl;
  if (c.dq.parts > 1) {
    use(a, c.dq);
    if (launch_k(la::xs::sum_rows_kernel<D, T>, dim3(unsigned(ceil_div(c.rows * (D / 2), la::xs::THREADS))), la::xs::THREADS, 0, st,
                 true, a, part, static_cast<T*>(dQ)))
      return LA_ERR_CUDA;
    ++*nl;
  }
  t.tiles = static_cast<int32_t>(ceil_div(p.Nk, la::xt::BN));
  t.splits = c.dkv.parts;
  t.per = c.dkv.per;
  t.total = p.B * p.Hkv * int64_t(t.tiles) * t.splits;
  divisions(p.Hkv);
  float* part_v = part + int64_t(c.dkv.parts) * c.keys * D;
  if (launch_k(kk, dim3(unsigned(std::min<int64_t>(t.total, sm))), la::xb::THREADS, mk, st, true, tq, tg, keys.k, keys.v, t,
               lse, delta, part, part_v))
    return LA_ERR_CUDA;
  if (launch_k(la::xs::sum_keys_kernel<D, T>, dim3(unsigned(ceil_div(c.keys * (D / 2), la::xs::THREADS)), 2), la::xs::THREADS, 0,
               st, true, c.keys, p.Hkv, p.Nk, c.dkv.parts, part, part_v,
               keys.count ? reinterpret_cast<const int32_t*>(ws + c.off_place) : static_cast<const int32_t*>(nullptr),
               static_cast<T*>(dK), static_cast<T*>(dV), a.dk, a.dv))
    return LA_ERR_CUDA;
  *nl += 2;
  return LA_OK;
}

template <typename F>
int with_type(const la_cross_problem& p, F&& f) {
  auto dim = [&](auto t) {
    switch (p.d) {
      case 32: return f(std::integral_constant<int, 32>(), t);
      case 64: return f(std::integral_constant<int, 64>(), t);
      default: return f(std::integral_constant<int, 128>(), t);
    }
  };
  return p.dtype == LA_BF16 ? dim(__nv_bfloat16()) : dim(float());
}

template <int D, typename T, int R>
int cross_few(const la_cross_problem& p, const CrossPlan& c, la::xs::Args a, const void* Q, const void* K, const void* V,
              void* O, float* lse, uint8_t* ws, cudaStream_t st, int* nl) {
  use(a, c.fwd);
  float* part_o = reinterpret_cast<float*>(ws + c.off_o);
  float2* part_ml = reinterpret_cast<float2*>(ws + c.off_ml);
  const size_t smem = la::xf::smem_bytes<D, R>();
  auto kern = la::xf::few_kernel<D, T, R>;
  if (set_smem(kern, smem)) return LA_ERR_CUDA;
  if (launch_k(kern, dim3(unsigned(p.B * p.Hkv * c.fwd.parts)), la::xf::THREADS, smem, st, false, a,
               static_cast<const T*>(Q), static_cast<const T*>(K), static_cast<const T*>(V), static_cast<T*>(O), lse, part_o,
               part_ml))
    return LA_ERR_CUDA;
  ++*nl;
  if (c.fwd.parts > 1) {
    if (launch_k(la::xs::join_kernel<D, T>, dim3(unsigned(c.rows)), 32 * la::xs::JOIN_WARPS, 0, st, true, a, part_o, part_ml, static_cast<T*>(O), lse))
      return LA_ERR_CUDA;
    ++*nl;
  }
  return LA_OK;
}

// Partial sums leave the kernels in 32-byte stores.  Workspaces have the 16-byte alignment of every
// pointer, so the parts start at the first 32-byte boundary, for which 16 bytes more are asked for.
constexpr size_t kCrossSlack = 16;

// The workspace of a call, from its first 32-byte boundary on.
int cross_workspace(const CrossPlan& c, void* ws, size_t ws_bytes, uint8_t** out) {
  const uintptr_t at = (reinterpret_cast<uintptr_t>(ws) + 31) & ~uintptr_t(31);
  *out = reinterpret_cast<uint8_t*>(at);
  if (!aligned16(ws)) return LA_ERR_ALIGN;
  if (c.total == 0) return LA_OK;
  const size_t skip = at - reinterpret_cast<uintptr_t>(ws);
  return ws && ws_bytes >= skip + c.total ? LA_OK : LA_ERR_WORKSPACE;
}

int need(const void* ptr, bool needed) {
  if (!needed) return LA_OK;
  if (!ptr) return LA_ERR_NULL;
  return aligned16(ptr) ? LA_OK : LA_ERR_ALIGN;
}

// Whether an output stands at the address of an input or of another output (null: not there).
template <size_t O, size_t I>
bool same_address(const void* const (&out)[O], const void* const (&in)[I]) {
  for (size_t i = 0; i < O; ++i) {
    if (!out[i]) continue;
    for (const void* x : in)
      if (x == out[i]) return true;
    for (size_t j = 0; j < i; ++j)
      if (out[j] == out[i]) return true;
  }
  return false;
}

// kv_len: 4-byte aligned.  (key_mask has no alignment.)
int check_len(const int32_t* kv_len) { return (reinterpret_cast<uintptr_t>(kv_len) & 3u) ? LA_ERR_ALIGN : LA_OK; }

// ------------------------------------------------------------------------------- layer norm
constexpr int64_t kMaxCols = 16384;
constexpr int64_t kFewRowsPerSm = 4;  // forward: up to here a block has one row

int validate(const la_norm_problem* p, bool backward) {
  if (!p) return LA_ERR_NULL;
  if (p->dtype != LA_BF16 && p->dtype != LA_F32) return LA_ERR_UNSUPPORTED;
  if (p->flags) return LA_ERR_UNSUPPORTED;
  if (p->rows < 0 || p->cols < 1 || p->cols > kMaxCols || p->groups < 1) return LA_ERR_SHAPE;
  if (p->rows > kMaxTokens || p->groups > kMaxTokens || p->rows % p->groups) return LA_ERR_SHAPE;
  if (!std::isfinite(p->eps) || p->eps < 0.f) return LA_ERR_SHAPE;
  if (double(p->groups) * double(p->cols) >= 1.0e12) return LA_ERR_SHAPE;
  const int64_t s[4] = {p->sx, p->sy, p->sdy, p->sdx};
  for (int i = 0; i < 4; ++i) {
    if (p->rows <= 1 || (backward ? i == 1 : i >= 2)) continue;
    if (s[i] < p->cols || double(s[i]) * double(p->rows) > 1.0e18) return LA_ERR_SHAPE;
  }
  return LA_OK;
}

// Whether rows of `in` (stride si) and of `out` (stride so) are the same rows or share no element.
bool norm_alias_ok(const la_norm_problem& p, const void* in, int64_t si, const void* out, int64_t so) {
  const int64_t e = int64_t(elem_size(p.dtype)), last = p.rows - 1;
  const int64_t a = reinterpret_cast<int64_t>(in), b = reinterpret_cast<int64_t>(out);
  if (last < 0) return true;
  if (a == b) return last == 0 || si == so;
  if (a + (last * si + p.cols) * e <= b || b + (last * so + p.cols) * e <= a) return true;
  if (last == 0 || si != so) return false;
  const int64_t s = si * e, d = ((b - a) % s + s) % s;  // columns of one buffer, side by side
  return d >= p.cols * e && d <= s - p.cols * e;
}

// Statistics, weights, biases and their gradients: dense fp32.  Whether one that is written shares an
// element with another one.
struct Floats {
  const float* at;
  int64_t n;
  bool output;
};
template <size_t N>
bool floats_overlap(const Floats (&f)[N]) {
  for (size_t i = 0; i < N; ++i)
    for (size_t j = 0; j < N; ++j) {
      if (i == j || !f[i].output || !f[i].at || !f[j].at || f[i].n == 0 || f[j].n == 0) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(f[i].at), b = reinterpret_cast<uintptr_t>(f[j].at);
      if (a < b + uintptr_t(f[j].n) * sizeof(float) && b < a + uintptr_t(f[i].n) * sizeof(float)) return true;
    }
  return false;
}

template <typename T>
bool norm_vec(const la_norm_problem& p, int n, const void* const* ptr, const int64_t* stride) {
  const int64_t vec = 16 / int64_t(sizeof(T));
  if (p.cols % vec) return false;
  for (int i = 0; i < n; ++i)
    if (!aligned16(ptr[i]) || (p.rows > 1 && stride[i] % vec)) return false;
  return true;
}

// Blocks per group (in the backward pass also slots of dweight and dbias): enough to fill the
// machine, each with at least 8 steps over its rows.
int norm_parts(const la_norm_problem& p, int sm, int per_sm) {
  const int64_t parts = int64_t(sm) * per_sm / std::max<int64_t>(p.groups, 1);
  return static_cast<int>(std::max<int64_t>(1, std::min(parts, ceil_div(p.rows / p.groups, 8))));
}
// Backward blocks that share an SM, by the registers of 16 elements a thread (a row, its weight and
// two sums for each): 2 blocks of 256 threads at 4096 columns, and in proportion.
int norm_backward_per_sm(int64_t cols) {
  return cols <= 512 ? 8 : cols <= 1024 ? 6 : cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1;
}

// The slots' bytes (they do not depend on the rows' alignment: every path fits).
size_t norm_slots(const la_norm_problem& p, int sm) {
  const int parts = norm_parts(p, sm, norm_backward_per_sm(p.cols));
  return parts > 1 ? align256(2 * size_t(p.groups) * size_t(parts) * size_t(p.cols) * 4) : 0;
}

// Ring stages: what lets as many blocks share an SM as there are, at least 1 and at most 4.
int norm_stages(size_t stage_bytes, int per_sm) {
  const size_t budget = (size_t(220) << 10) / size_t(per_sm);
  return static_cast<int>(std::max<size_t>(1, std::min<size_t>(4, budget / stage_bytes)));
}

struct NormForward {
  const void* x;
  const float *w, *b;
  void* y;
  float *mean, *rstd;
};

template <typename T, int VEC, int NV, int LPR, int U>
int norm_forward_short(const la_norm_problem&, const la::ln::Args& a, int, const NormForward& f, cudaStream_t st) {
  const int64_t rows = la::ln::WARPS * U * (32 / LPR);
  return launch_k(la::ln::forward_short<T, VEC, NV, LPR, U>, dim3(unsigned(ceil_div(a.rows, rows))), 32 * la::ln::WARPS, 0, st,
                  false, a, static_cast<const T*>(f.x), f.w, f.b, static_cast<T*>(f.y), f.mean, f.rstd);
}

template <typename T, int VEC, int NV, int WPR, bool RING>
int norm_forward_long(const la_norm_problem& p, const la::ln::Args& a, int sm, const NormForward& f, cudaStream_t st) {
  auto kern = la::ln::forward_long<T, VEC, NV, WPR, RING>;
  const int per_sm = WPR <= 8 ? 4 : 2;
  const int parts = p.rows <= kFewRowsPerSm * int64_t(sm) ? int(p.rows / p.groups) : norm_parts(p, sm, per_sm);
  const size_t row = size_t(p.cols) * sizeof(T);
  const int stages = RING ? norm_stages(row, per_sm) : 0;
  if (RING && set_smem(kern, stages * row)) return LA_ERR_CUDA;
  return launch_k(kern, dim3(unsigned(p.groups * parts)), 32 * WPR, stages * row, st, false, a, parts, stages,
                  static_cast<const T*>(f.x), f.w, f.b, static_cast<T*>(f.y), f.mean, f.rstd);
}

template <typename T>
int norm_forward_any(const la_norm_problem& p, const la::ln::Args& a, int sm, const NormForward& f, cudaStream_t st) {
  const void* ptr[2] = {f.x, f.y};
  const int64_t str[2] = {p.sx, p.sy};
  const int64_t c = p.cols;
  // Few rows do not fill the machine: what counts is how soon one is done, so more threads share it
  // (4096 channels of bf16, 64 rows: 2.5 us, a warp each 6.9; 600 rows: 7.1 and 7.7; 1200: 11.4 and 8.4).
  const bool few = p.rows <= kFewRowsPerSm * int64_t(sm);
  if (norm_vec<T>(p, 2, ptr, str)) {
    constexpr int V = 16 / int(sizeof(T));
    if (few && c > 32 * V && c <= 256 * V) return norm_forward_long<T, V, 1, 8, false>(p, a, sm, f, st);
    if (few && c > 256 * V && c <= 1024 * V) return norm_forward_long<T, V, 2, 16, false>(p, a, sm, f, st);
    if (c <= 8 * V) return norm_forward_short<T, V, 1, 8, 4>(p, a, sm, f, st);
    if (c <= 16 * V) return norm_forward_short<T, V, 1, 16, 4>(p, a, sm, f, st);
    if (c <= 32 * V) return norm_forward_short<T, V, 1, 32, 4>(p, a, sm, f, st);
    if (c <= 64 * V) return norm_forward_short<T, V, 2, 32, 2>(p, a, sm, f, st);
    if (c <= 128 * V) return norm_forward_short<T, V, 4, 32, 1>(p, a, sm, f, st);
    if (c <= 256 * V) return norm_forward_short<T, V, 8, 32, 1>(p, a, sm, f, st);
    if (c <= 512 * V) return norm_forward_short<T, V, 16, 32, 1>(p, a, sm, f, st);
    if (c <= 1024 * V) return norm_forward_long<T, V, 2, 16, true>(p, a, sm, f, st);
    if constexpr (2048 * V < kMaxCols)
      if (c > 2048 * V) return norm_forward_long<T, V, 8, 16, true>(p, a, sm, f, st);
    return norm_forward_long<T, V, 4, 16, true>(p, a, sm, f, st);
  }
  if (few && c > 32 * 4 && c <= 256 * 4) return norm_forward_long<T, 1, 4, 8, false>(p, a, sm, f, st);
  if (c <= 8 * 4) return norm_forward_short<T, 1, 4, 8, 2>(p, a, sm, f, st);
  if (c <= 32 * 4) return norm_forward_short<T, 1, 4, 32, 2>(p, a, sm, f, st);
  if (c <= 32 * 16) return norm_forward_short<T, 1, 16, 32, 1>(p, a, sm, f, st);
  if (c <= 32 * 32) return norm_forward_short<T, 1, 32, 32, 1>(p, a, sm, f, st);
  if (c <= 256 * 16) return norm_forward_long<T, 1, 16, 8, false>(p, a, sm, f, st);
  if (c <= 512 * 16) return norm_forward_long<T, 1, 16, 16, false>(p, a, sm, f, st);
  return norm_forward_long<T, 1, 32, 16, false>(p, a, sm, f, st);
}

struct NormGrads {
  const void *x, *dy;
  const float *w, *mean, *rstd;
  void* dx;
  float *dw, *db;  // or the slots
};

template <typename T, int VEC, int NV, int LPR, int U>
int norm_backward_short(const la::ln::Args& a, int64_t groups, int parts, const NormGrads& g, cudaStream_t st) {
  const size_t smem = g.dw || g.db ? size_t(la::ln::WARPS) * (32 / LPR) * size_t(a.cols) * 4 : 0;
  return launch_k(la::ln::backward_short<T, VEC, NV, LPR, U>, dim3(unsigned(groups * parts)), 32 * la::ln::WARPS, smem, st,
                  false, a, parts, static_cast<const T*>(g.x), static_cast<const T*>(g.dy), g.w, g.mean, g.rstd,
                  static_cast<T*>(g.dx), g.dw, g.db);
}

template <typename T, int VEC, int NV, int WPR, bool RING>
int norm_backward_long(const la::ln::Args& a, int64_t groups, int parts, const NormGrads& g, cudaStream_t st) {
  auto kern = la::ln::backward_long<T, VEC, NV, WPR, RING>;
  const size_t stage = 2 * size_t(a.cols) * sizeof(T);
  const int stages = RING ? norm_stages(stage, norm_backward_per_sm(a.cols)) : 0;
  if (RING && set_smem(kern, stages * stage)) return LA_ERR_CUDA;
  return launch_k(kern, dim3(unsigned(groups * parts)), 32 * WPR, stages * stage, st, false, a, parts, stages,
                  static_cast<const T*>(g.x), static_cast<const T*>(g.dy), g.w, g.mean, g.rstd, static_cast<T*>(g.dx), g.dw,
                  g.db);
}

template <typename T>
int norm_backward_any(const la_norm_problem& p, const la::ln::Args& a, int parts, const NormGrads& g, cudaStream_t st) {
  const void* ptr[3] = {g.x, g.dy, g.dx};
  const int64_t str[3] = {p.sx, p.sdy, p.sdx};
  const int64_t c = p.cols, n = p.groups;
  if (norm_vec<T>(p, 3, ptr, str)) {
    constexpr int V = 16 / int(sizeof(T));
    if (c <= 8 * V) return norm_backward_short<T, V, 1, 8, 2>(a, n, parts, g, st);
    if (c <= 16 * V) return norm_backward_short<T, V, 1, 16, 2>(a, n, parts, g, st);
    if (c <= 32 * V) return norm_backward_short<T, V, 1, 32, 2>(a, n, parts, g, st);
    if (c <= 512) return norm_backward_short<T, V, 16 / V, 32, 1>(a, n, parts, g, st);
    if (c <= 1024) return norm_backward_long<T, V, 16 / V, 2, true>(a, n, parts, g, st);
    if (c <= 2048) return norm_backward_long<T, V, 16 / V, 4, true>(a, n, parts, g, st);
    if (c <= 4096) return norm_backward_long<T, V, 16 / V, 8, true>(a, n, parts, g, st);
    if (c <= 8192) return norm_backward_long<T, V, 16 / V, 16, true>(a, n, parts, g, st);
    return norm_backward_long<T, V, 32 / V, 16, true>(a, n, parts, g, st);
  }
  if (c <= 8 * 4) return norm_backward_short<T, 1, 4, 8, 1>(a, n, parts, g, st);
  if (c <= 32 * 8) return norm_backward_short<T, 1, 8, 32, 1>(a, n, parts, g, st);
  if (c <= 256 * 8) return norm_backward_long<T, 1, 8, 8, false>(a, n, parts, g, st);
  if (c <= 256 * 16) return norm_backward_long<T, 1, 16, 8, false>(a, n, parts, g, st);
  if (c <= 512 * 16) return norm_backward_long<T, 1, 16, 16, false>(a, n, parts, g, st);
  return norm_backward_long<T, 1, 32, 16, false>(a, n, parts, g, st);
}

la::ln::Args norm_args(const la_norm_problem& p) {
  la::ln::Args a;
  a.rows = p.rows;
  a.per_group = p.rows / p.groups;
  a.sx = p.sx; a.sy = p.sy; a.sdy = p.sdy; a.sdx = p.sdx;
  a.cols = static_cast<int32_t>(p.cols);
  a.eps = p.eps;
  a.inv_cols = static_cast<float>(1.0 / double(p.cols));
  return a;
}

// ------------------------------------------------------------------------------- gradient clipping
constexpr int kClipCap = 1024;           // tensors per launch (the list rides in 32 KB of parameters)
constexpr int kClipBlocksPerSm = 8;

int64_t clip_tables(int64_t count) { return std::max<int64_t>(1, ceil_div(count, kClipCap)); }

size_t clip_need(int64_t count, int sm) { return align256(size_t(clip_tables(count)) * size_t(sm) * kClipBlocksPerSm * 8); }

int validate(const la_grad* g, int64_t count, bool clip) {
  if (count < 0 || count > (int64_t(1) << 24)) return LA_ERR_SHAPE;
  if (count > 0 && !g) return LA_ERR_NULL;
  double bytes = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].dtype != LA_BF16 && g[i].dtype != LA_F32) return LA_ERR_UNSUPPORTED;
    if (g[i].reserved) return LA_ERR_UNSUPPORTED;
    if (g[i].numel < 0) return LA_ERR_SHAPE;
    bytes += double(g[i].numel) * double(elem_size(g[i].dtype));
    if (bytes > 1.0e13) return LA_ERR_SHAPE;  // chunk numbers stay in 32 bits
    if (g[i].numel == 0) continue;
    const uintptr_t mask = elem_size(g[i].dtype) - 1;
    if (!g[i].in || (clip && !g[i].out)) return LA_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(g[i].in) & mask) || (clip && (reinterpret_cast<uintptr_t>(g[i].out) & mask)))
      return LA_ERR_ALIGN;
  }
  return LA_OK;
}

// Outputs (the norm too: it is written while gradients are still read) may overlap nothing but their own
// input at the same address.  One sweep over all ranges
// by rising start: an overlap shows between a range and the furthest end so far (kept for outputs
// and for inputs apart).
int clip_overlaps(const la_grad* g, int64_t count, const float* norm) {
  struct Range {
    uintptr_t a, b;
    bool out;
  };
  Range* r = new (std::nothrow) Range[size_t(2 * count + 1)];
  if (!r) return LA_ERR_SHAPE;
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].numel == 0) continue;
    const uintptr_t bytes = uintptr_t(g[i].numel) * elem_size(g[i].dtype);
    const uintptr_t o = reinterpret_cast<uintptr_t>(g[i].out), in = reinterpret_cast<uintptr_t>(g[i].in);
    r[n++] = {o, o + bytes, true};
    if (in != o) r[n++] = {in, in + bytes, false};  // (in place: the output's range stands for both)
  }
  auto before = [](const Range& x, const Range& y) { return x.a < y.a; };
  if (!std::is_sorted(r, r + n, before)) std::sort(r, r + n, before);
  const uintptr_t at = reinterpret_cast<uintptr_t>(norm);  // (apart, so that lists in order stay in order)
  uintptr_t end_out = 0, end_in = 0;
  int rc = LA_OK;
  for (int64_t i = 0; i < n && rc == LA_OK; ++i) {
    if (r[i].a < end_out || (r[i].out && r[i].a < end_in)) rc = LA_ERR_SHAPE;
    if (r[i].a < at + sizeof(float) && at < r[i].b) rc = LA_ERR_SHAPE;
    uintptr_t& end = r[i].out ? end_out : end_in;
    end = std::max(end, r[i].b);
  }
  delete[] r;
  return rc;
}

template <int CAP>
int64_t fill_table(la::clip::Table<CAP>& t, const la_grad* g, int64_t count) {
  std::memset(t.f32, 0, sizeof t.f32);
  int n = 0;
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].numel == 0) continue;
    const int64_t per = la::clip::CHUNK_BYTES / int64_t(elem_size(g[i].dtype));
    t.in[n] = g[i].in;
    t.out[n] = g[i].out;
    t.numel[n] = g[i].numel;
    t.chunk0[n] = static_cast<uint32_t>(chunks);
    if (g[i].dtype == LA_F32) t.f32[n >> 5] |= 1u << (n & 31);
    chunks += ceil_div(g[i].numel, per);
    ++n;
  }
  t.count = n;
  t.chunks = static_cast<uint32_t>(chunks);
  return chunks;
}

template <int CAP>
int clip_norm_launch(const la_grad* g, int64_t count, int max_blocks, double* partial, int* parts, cudaStream_t st, int* nl) {
  la::clip::Table<CAP> t;
  const int64_t chunks = fill_table(t, g, count);
  if (chunks == 0) return LA_OK;
  const int64_t blocks = std::min<int64_t>(chunks, max_blocks);
  if (launch_k(la::clip::norm_kernel<CAP>, dim3(unsigned(blocks)), la::clip::THREADS, 0, st, false, t, partial + *parts))
    return LA_ERR_CUDA;
  *parts += static_cast<int>(blocks);
  ++*nl;
  return LA_OK;
}

template <int CAP>
int clip_scale_launch(const la_grad* g, int64_t count, int max_blocks, const double* partial, int parts, float max_norm,
                      float* norm, cudaStream_t st, int* nl) {
  la::clip::Table<CAP> t;
  const int64_t chunks = fill_table(t, g, count);
  if (chunks == 0) return LA_OK;
  const int64_t blocks = std::min<int64_t>(chunks, max_blocks);
  if (launch_k(la::clip::scale_kernel<CAP>, dim3(unsigned(blocks)), la::clip::THREADS, 0, st, true, t, partial, parts,
               max_norm, norm))
    return LA_ERR_CUDA;
  ++*nl;
  return LA_OK;
}

int clip_common(const la_grad* g, int64_t count, bool clip, float max_norm, float* norm, void* ws, size_t ws_bytes,
                cudaStream_t st) {
  int rc = validate(g, count, clip);
  if (rc) return rc;
  if (!norm) return LA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(norm) & 3u) return LA_ERR_ALIGN;
  if (clip && (!std::isfinite(max_norm) || max_norm < 0.f)) return LA_ERR_SHAPE;
  if (clip && (rc = clip_overlaps(g, count, norm))) return rc;
  int sm = 0;
  if ((rc = current_sm_count(&sm))) return rc;
  if (!ws || ws_bytes < clip_need(count, sm)) return LA_ERR_WORKSPACE;
  if (!aligned16(ws)) return LA_ERR_ALIGN;
  double* partial = static_cast<double*>(ws);
  const int blocks = sm * kClipBlocksPerSm;
  int nl = 0, parts = 0;
  // The smallest table that holds a list: launch parameters cost time by their size.
  auto each = [&](auto&& f) {
    for (int64_t i = 0; i < count; i += kClipCap) {
      const int64_t n = std::min<int64_t>(kClipCap, count - i);
      const int r = n <= 32 ? f(std::integral_constant<int, 32>(), g + i, n)
                            : n <= 256 ? f(std::integral_constant<int, 256>(), g + i, n)
                                       : f(std::integral_constant<int, kClipCap>(), g + i, n);
      if (r) return r;
    }
    return int(LA_OK);
  };
  if ((rc = each([&](auto cap, const la_grad* p, int64_t n) {
         return clip_norm_launch<decltype(cap)::value>(p, n, blocks, partial, &parts, st, &nl);
       })))
    return rc;
  if (clip && parts > 0) {
    float* out = norm;
    if ((rc = each([&](auto cap, const la_grad* p, int64_t n) {
           const int before = nl;
           const int r = clip_scale_launch<decltype(cap)::value>(p, n, blocks, partial, parts, max_norm, out, st, &nl);
           if (nl > before) out = nullptr;  // the first launch writes the norm
           return r;
         })))
      return rc;
  } else {
    if (launch_k(la::clip::finish_kernel, dim3(1), la::clip::THREADS, 0, st, parts > 0, partial, parts, norm)) return LA_ERR_CUDA;
    ++nl;
  }
  g_last_launches = nl;
  return LA_OK;
}

}  // namespace

extern "C" {

size_t la_cross_workspace_bytes_of(const la_cross_problem* p, unsigned uses, int sm_count) {
  if (validate(p, false) != LA_OK || sm_count < 0 || (uses & ~unsigned(LA_CROSS_ANY))) return 0;
  if (sm_count == 0 && current_sm_count(&sm_count) != LA_OK) return 0;
  const unsigned forward = uses & ~unsigned(LA_CROSS_BACKWARD), backward = uses & ~unsigned(LA_CROSS_FORWARD);
  size_t total = 0;
  if (uses & LA_CROSS_FORWARD) total = cross_plan(*p, sm_count, forward).total;
  if (uses & LA_CROSS_BACKWARD) total = std::max(total, cross_plan(*p, sm_count, backward).total);
  return total + kCrossSlack;
}

size_t la_cross_workspace_bytes_for(const la_cross_problem* p, int sm_count) {
  return sm_count > 0 ? la_cross_workspace_bytes_of(p, LA_CROSS_ANY, sm_count) : 0;
}

size_t la_cross_workspace_bytes(const la_cross_problem* p) { return la_cross_workspace_bytes_of(p, LA_CROSS_ANY, 0); }

int la_cross_forward(const la_cross_problem* p, const void* Q, const void* K, const void* V, const int32_t* kv_len,
                     const uint8_t* key_mask, void* O, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = validate(p, false);
  if (rc) return rc;
  const bool has_q = p->B * p->H > 0 && p->Nq > 0, has_k = has_q && p->Nk > 0;
  if ((rc = need(Q, has_q)) || (rc = need(K, has_k)) || (rc = need(V, has_k)) || (rc = need(O, has_q)) ||
      (rc = need(lse, has_q && lse)) || (rc = check_len(kv_len)))
    return rc;
  // (O and lse are written as the rest is read; K and V of no keys have no address)
  if (has_q && same_address({O, lse}, {Q, has_k ? K : nullptr, has_k ? V : nullptr, kv_len, key_mask})) return LA_ERR_SHAPE;
  int sm = 0;
  if ((rc = current_sm_count(&sm))) return rc;
  const CrossPlan c = cross_plan(*p, sm, uses_of(LA_CROSS_FORWARD, kv_len, key_mask));
  uint8_t* w = nullptr;
  if ((rc = cross_workspace(c, ws, ws_bytes, &w))) return rc;
  int nl = 0;
  if (has_q) {
    const la::xs::Args a = cross_args(*p, c, kv_len, key_mask);
    rc = with_type(*p, [&](auto d, auto t) {
      constexpr int D = decltype(d)::value;
      using T = decltype(t);
      if (c.few) {
        const int64_t r = p->H / p->Hkv * p->Nq;
        auto f = r <= 1 ? cross_few<D, T, 1> : r <= 2 ? cross_few<D, T, 2> : r <= 4 ? cross_few<D, T, 4> : cross_few<D, T, 8>;
        return f(*p, c, a, Q, K, V, O, lse, w, stream, &nl);
      }
      if constexpr (sizeof(t) == 2) {
        if (c.tc) return cross_forward_tc<D>(*p, c, a, Q, K, V, O, lse, w, sm, stream, &nl);
      }
      return cross_forward_simt<D, decltype(t)>(*p, c, a, Q, K, V, O, lse, w, stream, &nl);
    });
    if (rc) return rc;
  }
  g_last_launches = nl;
  return LA_OK;
}

int la_cross_backward(const la_cross_problem* p, const void* Q, const void* K, const void* V, const int32_t* kv_len,
                      const uint8_t* key_mask, const void* O, const float* lse, const void* dO, void* dQ, void* dK,
                      void* dV, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = validate(p, true);
  if (rc) return rc;
  const bool has_q = p->B * p->H > 0 && p->Nq > 0, has_k = p->B * p->H > 0 && p->Nk > 0;
  if ((rc = need(Q, has_q)) || (rc = need(K, has_k)) || (rc = need(V, has_k)) || (rc = need(O, has_q)) ||
      (rc = need(lse, has_q)) || (rc = need(dO, has_q)) || (rc = need(dQ, has_q)) || (rc = need(dK, has_k)) ||
      (rc = need(dV, has_k)) || (rc = check_len(kv_len)))
    return rc;
  // (an input is read after the first gradient is written)
  auto here = [](const void* x, bool has) { return has ? x : nullptr; };
  if (same_address({here(dQ, has_q), here(dK, has_k), here(dV, has_k)},
                   {here(Q, has_q), here(K, has_k), here(V, has_k), here(O, has_q), static_cast<const void*>(here(lse, has_q)),
                    here(dO, has_q), kv_len, key_mask}))
    return LA_ERR_SHAPE;
  int sm = 0;
  if ((rc = current_sm_count(&sm))) return rc;
  const CrossPlan c = cross_plan(*p, sm, uses_of(LA_CROSS_BACKWARD, kv_len, key_mask));
  uint8_t* w = nullptr;
  if ((rc = cross_workspace(c, ws, ws_bytes, &w))) return rc;
  int nl = 0;
  const la::xs::Args a = cross_args(*p, c, kv_len, key_mask);
  rc = with_type(*p, [&](auto d, auto t) {
    constexpr int D = decltype(d)::value;
    if constexpr (sizeof(t) == 2) {
      if (c.tc) return cross_backward_tc<D>(*p, c, a, Q, K, V, O, lse, dO, dQ, dK, dV, w, sm, stream, &nl);
    }
    return cross_backward_simt<D, decltype(t)>(*p, c, a, Q, K, V, O, lse, dO, dQ, dK, dV, w, stream, &nl);
  });
  if (rc) return rc;
  g_last_launches = nl;
  return LA_OK;
}

size_t la_layernorm_workspace_bytes_for(const la_norm_problem* p, int sm_count) {
  if (validate(p, false) != LA_OK || sm_count <= 0) return 0;
  return std::max<size_t>(norm_slots(*p, sm_count), 16);
}

size_t la_layernorm_workspace_bytes(const la_norm_problem* p) {
  int sm = 0;
  if (validate(p, false) != LA_OK || current_sm_count(&sm) != LA_OK) return 0;
  return la_layernorm_workspace_bytes_for(p, sm);
}

int la_layernorm_forward(const la_norm_problem* p, const void* x, const float* weight, const float* bias, void* y,
                         float* mean, float* rstd, cudaStream_t stream) {
  int rc = validate(p, false);
  if (rc) return rc;
  const bool has = p->rows > 0;
  if (has && (!x || !y || !mean != !rstd)) return LA_ERR_NULL;
  const uintptr_t mask = elem_size(p->dtype) - 1;
  if ((reinterpret_cast<uintptr_t>(x) & mask) || (reinterpret_cast<uintptr_t>(y) & mask)) return LA_ERR_ALIGN;
  if (!aligned16(weight) || !aligned16(bias) || !aligned16(mean) || !aligned16(rstd)) return LA_ERR_ALIGN;
  if (has && !norm_alias_ok(*p, x, p->sx, y, p->sy)) return LA_ERR_SHAPE;
  const int64_t params = p->groups * p->cols;
  if (floats_overlap({{weight, params, false}, {bias, params, false}, {mean, p->rows, true}, {rstd, p->rows, true}}) ||
      (has && (same_address({y}, {weight, bias}) || same_address({mean, rstd}, {x, y}))))
    return LA_ERR_SHAPE;
  if (has) {
    int sm = 0;
    if ((rc = current_sm_count(&sm))) return rc;
    const la::ln::Args a = norm_args(*p);
    const NormForward f = {x, weight, bias, y, mean, rstd};
    rc = p->dtype == LA_BF16 ? norm_forward_any<__nv_bfloat16>(*p, a, sm, f, stream) : norm_forward_any<float>(*p, a, sm, f, stream);
    if (rc) return rc;
  }
  g_last_launches = has ? 1 : 0;
  return LA_OK;
}

int la_layernorm_backward(const la_norm_problem* p, const void* x, const void* dy, const float* weight, const float* mean,
                          const float* rstd, void* dx, float* dweight, float* dbias, void* ws, size_t ws_bytes,
                          cudaStream_t stream) {
  int rc = validate(p, true);
  if (rc) return rc;
  const bool has = p->rows > 0;
  if (has && (!x || !dy || !dx || !mean || !rstd)) return LA_ERR_NULL;
  const uintptr_t mask = elem_size(p->dtype) - 1;
  for (const void* t : {x, dy, static_cast<const void*>(dx)})
    if (reinterpret_cast<uintptr_t>(t) & mask) return LA_ERR_ALIGN;
  for (const float* t : {weight, mean, rstd, static_cast<const float*>(dweight), static_cast<const float*>(dbias)})
    if (!aligned16(t)) return LA_ERR_ALIGN;
  if (has && (!norm_alias_ok(*p, x, p->sx, dx, p->sdx) || !norm_alias_ok(*p, dy, p->sdy, dx, p->sdx))) return LA_ERR_SHAPE;
  const int64_t params = p->groups * p->cols;
  if (floats_overlap({{weight, params, false}, {mean, p->rows, false}, {rstd, p->rows, false}, {dweight, params, true},
                      {dbias, params, true}}) ||
      (has && (same_address({dx}, {weight, mean, rstd}) || same_address({dweight, dbias}, {x, dy, dx}))))
    return LA_ERR_SHAPE;
  int sm = 0;
  if ((rc = current_sm_count(&sm))) return rc;
  const size_t need_bytes = norm_slots(*p, sm);
  const int parts = norm_parts(*p, sm, norm_backward_per_sm(p->cols));
  const bool grads = dweight || dbias;
  if (grads && need_bytes > 0 && (!ws || ws_bytes < need_bytes)) return LA_ERR_WORKSPACE;
  if (!aligned16(ws)) return LA_ERR_ALIGN;
  int nl = 0;
  if (!has) {
    // no rows: the sums are 0 (the parts' slots are not used)
    const size_t bytes = size_t(p->groups) * size_t(p->cols) * 4;
    if (dweight && cudaMemsetAsync(dweight, 0, bytes, stream) != cudaSuccess) return LA_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, bytes, stream) != cudaSuccess) return LA_ERR_CUDA;
    g_last_launches = 0;
    return LA_OK;
  }
  const la::ln::Args a = norm_args(*p);
  const bool slots = grads && parts > 1;
  float* s_dw = static_cast<float*>(ws);
  float* s_db = s_dw + p->groups * int64_t(parts) * p->cols;
  const NormGrads g = {x, dy, weight, mean, rstd, dx, slots ? (dweight ? s_dw : nullptr) : dweight,
                       slots ? (dbias ? s_db : nullptr) : dbias};
  rc = p->dtype == LA_BF16 ? norm_backward_any<__nv_bfloat16>(*p, a, parts, g, stream)
                           : norm_backward_any<float>(*p, a, parts, g, stream);
  if (rc) return rc;
  ++nl;
  if (slots) {
    const int64_t blocks = p->groups * ceil_div(p->cols, la::ln::RED_COLS);
    if (launch_k(la::ln::reduce_kernel, dim3(unsigned(blocks), 2), la::ln::RED_COLS * la::ln::RED_ROWS, 0, stream, true, p->cols,
                 parts, s_dw, s_db, dweight, dbias))
      return LA_ERR_CUDA;
    ++nl;
  }
  g_last_launches = nl;
  return LA_OK;
}

size_t la_clip_workspace_bytes_for(int64_t count, int sm_count) {
  if (count < 0 || count > (int64_t(1) << 24) || sm_count <= 0) return 0;
  return clip_need(count, sm_count);
}

size_t la_clip_workspace_bytes(int64_t count) {
  int sm = 0;
  if (current_sm_count(&sm) != LA_OK) return 0;
  return la_clip_workspace_bytes_for(count, sm);
}

int la_grad_norm(const la_grad* grads, int64_t count, float* norm, void* ws, size_t ws_bytes, cudaStream_t stream) {
  return clip_common(grads, count, false, 0.f, norm, ws, ws_bytes, stream);
}

int la_clip_grad_norm(const la_grad* grads, int64_t count, float max_norm, float* norm, void* ws, size_t ws_bytes,
                      cudaStream_t stream) {
  return clip_common(grads, count, true, max_norm, norm, ws, ws_bytes, stream);
}

#ifdef LA_TEST_HOOKS
// Hooks build only (not part of the regular library): what is held back or lost from the next launch on
// (HOLD_*, LOSE_* in sm100.cuh; 0: nothing).
int la_test_hooks(unsigned int what) {
  return cudaMemcpyToSymbol(la::g_la_hooks, &what, sizeof what) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}
#endif

}  // extern "C"
