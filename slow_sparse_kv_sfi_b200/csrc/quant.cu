// 8-bit paged cache: pages of 16 tokens as e4m3 or int8 codes with one scale
// per (page, KV head) for the keys and one for the values, and the block index
// (int8 bounds of every page's keys).
//
// One warp moves one (page, KV head) of K or of V.  Its 16 rows are one
// contiguous run of 16 * D values, read whole into registers (16 bytes per
// lane and load, all loads issued before the first use), so every value is read
// once; the page's maximum is a warp reduction, and codes, scale and bounds
// leave from registers.  Bound by memory: 4 D bytes in and 2 D + small out per
// (token, KV head) for a store, the reverse for a load.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace sfi {
namespace {

constexpr float kAmaxFloor = 7.888609052210118e-31f;   // 2^-100: smaller pages share this scale
constexpr int kNoFormat = -1;                          // bounds only

struct QuantArgs {
  int B, Hkv, L, num_pages, max_pages;
  int page_lo;                 // first page of the range
  const int32_t* lens;
  // bf16 cache (source of a store, target of a load)
  const int32_t* pt;
  __nv_bfloat16* k_pool;
  __nv_bfloat16* v_pool;
  // 8-bit cache
  const int32_t* qpt;
  uint8_t* kq;
  uint8_t* vq;
  float* ks;
  float* vs;
  __nv_bfloat16* k_tail;
  __nv_bfloat16* v_tail;
  // block index
  const int32_t* ipt;
  int8_t* bounds;
  float* bscale;
  // appended token
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  int* err;
  int* err_kv;    // of the bf16 cache
  int* err_ix;    // of the index
};

// Lane layout of a page: CH lanes cover a row with 8 values each, RPI rows per
// load, NI loads.
template <int D>
struct Lay {
  static constexpr int CH = D / 8, RPI = 32 / CH, NI = 16 / RPI;
};

__device__ __forceinline__ float2 bf2(uint32_t v) { return unpack_bf16x2(v); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int sh = 16; sh >= 1; sh >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, sh));
  return v;
}

// NaN -> 0, +-infinity -> +-largest finite bf16.
__device__ __forceinline__ float tame(float x) {
  const float big = __uint_as_float(0x7f7f0000u);
  return x != x ? 0.f : fminf(fmaxf(x, -big), big);
}

// Codes and scale of the page in x (this lane's 8 values of NI rows).
template <int D, int FMT>
__device__ __forceinline__ void write_codes(const uint4 (&x)[Lay<D>::NI], int lane, uint8_t* codes, float* scale) {
  using Y = Lay<D>;
  uint32_t amax2 = 0;   // bf16x2 magnitudes compare as integers; NaN and infinity are the largest
#pragma unroll
  for (int i = 0; i < Y::NI; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) amax2 = __vmaxu2(amax2, w[j] & 0x7fff7fffu);
  }
  uint32_t am = max(amax2 & 0xffffu, amax2 >> 16);
#pragma unroll
  for (int sh = 16; sh >= 1; sh >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, sh));
  const bool finite = am < 0x7f80u;
  const float amax = fmaxf(__uint_as_float(am << 16), kAmaxFloor);
  constexpr float Q = FMT == SFI_FMT_E4M3 ? 448.f : 127.f;
  const float inv = __fdiv_rn(Q, amax);
  if (lane == 0) *scale = finite ? __fdiv_rn(amax, Q) : __uint_as_float(0x7fc00000u);
  const int row0 = lane / Y::CH, ch = lane % Y::CH;
#pragma unroll
  for (int i = 0; i < Y::NI; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 a = bf2(w[2 * j]), b = bf2(w[2 * j + 1]);
      uint32_t r;
      if constexpr (FMT == SFI_FMT_E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a.x * inv, a.y * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(b.x * inv, b.y * inv), __NV_SATFINITE, __NV_E4M3);
        r = lo | (hi << 16);
      } else {
        const int c0 = __float2int_rn(a.x * inv), c1 = __float2int_rn(a.y * inv);
        const int c2 = __float2int_rn(b.x * inv), c3 = __float2int_rn(b.y * inv);
        r = (c0 & 255) | ((c1 & 255) << 8) | ((c2 & 255) << 16) | ((uint32_t)(c3 & 255) << 24);
      }
      o[j] = finite ? r : 0u;
    }
    *reinterpret_cast<uint2*>(codes + (size_t)(i * Y::RPI + row0) * D + ch * 8) = make_uint2(o[0], o[1]);
  }
}

// Bounds of the page in x: per dimension the largest and smallest key, over
// the page's power-of-two scale, rounded outwards.
template <int D>
__device__ __forceinline__ void write_bounds(const uint4 (&x)[Lay<D>::NI], int lane, int8_t* bounds, float* scale) {
  using Y = Lay<D>;
  float hi[8], lo[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    hi[e] = -INFINITY;
    lo[e] = INFINITY;
  }
#pragma unroll
  for (int i = 0; i < Y::NI; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = bf2(w[j]);
      const float u = tame(a.x), v = tame(a.y);
      hi[2 * j] = fmaxf(hi[2 * j], u);
      lo[2 * j] = fminf(lo[2 * j], u);
      hi[2 * j + 1] = fmaxf(hi[2 * j + 1], v);
      lo[2 * j + 1] = fminf(lo[2 * j + 1], v);
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int sh = Y::CH; sh < 32; sh <<= 1) {
      hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], sh));
      lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], sh));
    }
    amax = fmaxf(amax, fmaxf(fabsf(hi[e]), fabsf(lo[e])));
  }
  amax = warp_max(amax);
  const int e = unit_exponent(amax);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
  if (lane == 0) *scale = __uint_as_float((uint32_t)(e + 127) << 23);
  if (lane < Y::CH) {
    uint32_t ph[2] = {0u, 0u}, pl[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      ph[k / 4] |= (uint32_t)((int)ceilf(hi[k] * inv) & 255) << (8 * (k % 4));
      pl[k / 4] |= (uint32_t)((int)floorf(lo[k] * inv) & 255) << (8 * (k % 4));
    }
    *reinterpret_cast<uint2*>(bounds + lane * 8) = make_uint2(ph[0], ph[1]);
    *reinterpret_cast<uint2*>(bounds + D + lane * 8) = make_uint2(pl[0], pl[1]);
  }
}

// The page of sequence b at index p through table pt, or -1 (latched).
__device__ __forceinline__ int page_of(const QuantArgs& a, const int32_t* pt, int b, int p, int lane, int* err) {
  const int page = pt[(size_t)b * a.max_pages + p];
  if ((unsigned)page < (unsigned)a.num_pages) return page;
  if (lane == 0) latch_error(err, SFI_ERR_DEVICE_CHECK, kSiteQuantPage);
  return -1;
}

// Work unit u of the range kernels: (sequence, page, KV head, K or V).
struct Unit {
  int b, p, h, v;
};
__device__ __forceinline__ Unit unit_of(long u, int n_pages, int Hkv, int nkv) {
  Unit r;
  r.v = (int)(u % nkv);
  u /= nkv;
  r.h = (int)(u % Hkv);
  u /= Hkv;
  r.p = (int)(u % n_pages);
  r.b = (int)(u / n_pages);
  return r;
}

// Store: bf16 pages [page_lo, ...) of every sequence -> codes, scales, bounds;
// the page that is not full -> tail.  FMT == kNoFormat: bounds only.
template <int D, int FMT>
__global__ void __launch_bounds__(256) store_kernel(const QuantArgs a, int n_pages, long units) {
  grid_dep_enter_writer();
  using Y = Lay<D>;
  const int lane = threadIdx.x & 31;
  const long u = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (u >= units) return;
  const Unit w = unit_of(u, n_pages, a.Hkv, FMT == kNoFormat ? 1 : 2);
  const int len = seq_len(a.lens, a.L, w.b, a.err);
  const int p = a.page_lo + w.p;
  const int rows = min(kPage, len - p * kPage);
  if (rows <= 0 || (FMT == kNoFormat && rows < kPage)) return;
  const int src = page_of(a, a.pt, w.b, p, lane, a.err_kv);
  if (src < 0) return;
  const __nv_bfloat16* from = (w.v ? a.v_pool : a.k_pool) + ((size_t)src * a.Hkv + w.h) * (kPage * D);
  const int row0 = lane / Y::CH, ch = lane % Y::CH;
  uint4 x[Y::NI];
#pragma unroll
  for (int i = 0; i < Y::NI; ++i) {
    const int r = i * Y::RPI + row0;
    x[i] = r < rows ? __ldg(reinterpret_cast<const uint4*>(from + r * D + ch * 8)) : make_uint4(0, 0, 0, 0);
  }
  if (rows < kPage) {
    __nv_bfloat16* tail = (w.v ? a.v_tail : a.k_tail) + ((size_t)w.b * a.Hkv + w.h) * (kPage * D);
#pragma unroll
    for (int i = 0; i < Y::NI; ++i) {
      const int r = i * Y::RPI + row0;
      if (r < rows) *reinterpret_cast<uint4*>(tail + r * D + ch * 8) = x[i];
    }
    return;
  }
  if constexpr (FMT != kNoFormat) {
    const int dst = page_of(a, a.qpt, w.b, p, lane, a.err);
    if (dst >= 0) {
      const size_t ph = (size_t)dst * a.Hkv + w.h;
      write_codes<D, FMT>(x, lane, (w.v ? a.vq : a.kq) + ph * (kPage * D), (w.v ? a.vs : a.ks) + ph);
    }
  }
  if (a.bounds && !w.v) {
    const int ip = page_of(a, a.ipt, w.b, p, lane, a.err_ix);
    if (ip >= 0) {
      const size_t ph = (size_t)ip * a.Hkv + w.h;
      write_bounds<D>(x, lane, a.bounds + ph * 2 * D, a.bscale + ph);
    }
  }
}

// Append: one token of every (sequence, KV head), K or V per warp.
template <int D, int FMT>
__global__ void __launch_bounds__(128) append_quant_kernel(const QuantArgs a, int units) {
  grid_dep_enter_writer();
  using Y = Lay<D>;
  const int lane = threadIdx.x & 31;
  const int u = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (u >= units) return;
  const int v = u & 1, bh = u >> 1, b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int len = seq_len(a.lens, a.L, b, a.err);
  if (len < 1) return;
  const int p = (len - 1) / kPage, row = (len - 1) % kPage;
  const __nv_bfloat16* tok = (v ? a.v_new : a.k_new) + (size_t)bh * D;
  __nv_bfloat16* tail = (v ? a.v_tail : a.k_tail) + (size_t)bh * (kPage * D);
  const int row0 = lane / Y::CH, ch = lane % Y::CH;
  const uint4 t = __ldg(reinterpret_cast<const uint4*>(tok + ch * 8));
  if (row == kPage - 1) {
    // the page is full: its first 15 rows come from the tail, the last is the token
    uint4 x[Y::NI];
#pragma unroll
    for (int i = 0; i < Y::NI; ++i) {
      const int r = i * Y::RPI + row0;
      x[i] = r < kPage - 1 ? *reinterpret_cast<const uint4*>(tail + r * D + ch * 8) : t;
    }
    const int dst = page_of(a, a.qpt, b, p, lane, a.err);
    if (dst >= 0) {
      const size_t ph = (size_t)dst * a.Hkv + h;
      write_codes<D, FMT>(x, lane, (v ? a.vq : a.kq) + ph * (kPage * D), (v ? a.vs : a.ks) + ph);
    }
    if (a.bounds && !v) {
      const int ip = page_of(a, a.ipt, b, p, lane, a.err_ix);
      if (ip >= 0) {
        const size_t ph = (size_t)ip * a.Hkv + h;
        write_bounds<D>(x, lane, a.bounds + ph * 2 * D, a.bscale + ph);
      }
    }
  }
  if (row0 == 0) *reinterpret_cast<uint4*>(tail + row * D + ch * 8) = t;
}

__device__ __forceinline__ uint32_t decode2(uint32_t codes, float scale, int fmt) {   // two codes -> bf16x2
  float2 f;
  if (fmt == SFI_FMT_E4M3) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3);
    f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  } else {
    f = make_float2((float)(int8_t)(codes & 255u), (float)(int8_t)((codes >> 8) & 255u));
  }
  return pack_bf16x2(f.x * scale, f.y * scale);
}

// Load: the 8-bit pages and the tail -> bf16 pages.
template <int D, int FMT>
__global__ void __launch_bounds__(256) load_kernel(const QuantArgs a, int n_pages, long units) {
  grid_dep_enter_writer();
  using Y = Lay<D>;
  const int lane = threadIdx.x & 31;
  const long u = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (u >= units) return;
  const Unit w = unit_of(u, n_pages, a.Hkv, 2);
  const int len = seq_len(a.lens, a.L, w.b, a.err);
  const int p = a.page_lo + w.p;
  const int rows = min(kPage, len - p * kPage);
  if (rows <= 0) return;
  const int dst = page_of(a, a.pt, w.b, p, lane, a.err_kv);
  if (dst < 0) return;
  __nv_bfloat16* to = (w.v ? a.v_pool : a.k_pool) + ((size_t)dst * a.Hkv + w.h) * (kPage * D);
  const int row0 = lane / Y::CH, ch = lane % Y::CH;
  if (rows < kPage) {
    const __nv_bfloat16* tail = (w.v ? a.v_tail : a.k_tail) + ((size_t)w.b * a.Hkv + w.h) * (kPage * D);
#pragma unroll
    for (int i = 0; i < Y::NI; ++i) {
      const int r = i * Y::RPI + row0;
      if (r < rows)
        *reinterpret_cast<uint4*>(to + r * D + ch * 8) = __ldg(reinterpret_cast<const uint4*>(tail + r * D + ch * 8));
    }
    return;
  }
  const int src = page_of(a, a.qpt, w.b, p, lane, a.err);
  if (src < 0) return;
  const size_t ph = (size_t)src * a.Hkv + w.h;
  const uint8_t* from = (w.v ? a.vq : a.kq) + ph * (kPage * D);
  const float scale = __ldg((w.v ? a.vs : a.ks) + ph);
  uint2 x[Y::NI];
#pragma unroll
  for (int i = 0; i < Y::NI; ++i)
    x[i] = __ldg(reinterpret_cast<const uint2*>(from + (i * Y::RPI + row0) * D + ch * 8));
#pragma unroll
  for (int i = 0; i < Y::NI; ++i)
    *reinterpret_cast<uint4*>(to + (i * Y::RPI + row0) * D + ch * 8) =
        make_uint4(decode2(x[i].x, scale, FMT), decode2(x[i].x >> 16, scale, FMT), decode2(x[i].y, scale, FMT),
                   decode2(x[i].y >> 16, scale, FMT));
}

QuantArgs base_args(const sfi_shape& s, int pos_lo, int L, const int32_t* lens) {
  QuantArgs a{};
  a.B = s.B;
  a.Hkv = s.Hkv;
  a.L = L;
  a.num_pages = s.num_pages;
  a.max_pages = s.max_pages;
  a.page_lo = pos_lo / kPage;
  a.lens = lens;
  return a;
}

void add_kv(QuantArgs& a, const sfi_paged_kv& kv) {
  a.pt = kv.page_table;
  a.k_pool = reinterpret_cast<__nv_bfloat16*>(kv.k_pool);
  a.v_pool = reinterpret_cast<__nv_bfloat16*>(kv.v_pool);
  a.err_kv = kv.err;
}

void add_quant(QuantArgs& a, const sfi_quant_kv& q) {
  a.qpt = q.page_table;
  a.kq = q.k_pool;
  a.vq = q.v_pool;
  a.ks = q.k_scale;
  a.vs = q.v_scale;
  a.k_tail = reinterpret_cast<__nv_bfloat16*>(q.k_tail);
  a.v_tail = reinterpret_cast<__nv_bfloat16*>(q.v_tail);
  a.err = q.err;
}

void add_index(QuantArgs& a, const sfi_block_index* ix) {
  if (!ix) return;
  a.ipt = ix->page_table;
  a.bounds = ix->bounds;
  a.bscale = ix->scale;
  a.err_ix = ix->err;
}

sfi_status check_range(const sfi_shape* s, int pos_lo, int L) {
  if (L < 0 || L > s->max_pages * kPage) return SFI_ERR_SHAPE;
  if (pos_lo < 0 || pos_lo % kPage != 0) return SFI_ERR_SHAPE;
  return SFI_OK;
}

sfi_status launched(cudaError_t e) {
  if (e == cudaSuccess) return SFI_OK;
  cudaGetLastError();
  return SFI_ERR_CUDA;
}

#define SFI_TRY(x)               \
  do {                           \
    sfi_status _r = (x);         \
    if (_r != SFI_OK) return _r; \
  } while (0)

}  // namespace

sfi_status check_quant(const sfi_quant_kv* q) {
  if (!q || !q->k_pool || !q->v_pool || !q->k_scale || !q->v_scale || !q->k_tail || !q->v_tail || !q->page_table)
    return SFI_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(q->k_pool) | reinterpret_cast<uintptr_t>(q->v_pool)) & 31u) != 0)
    return SFI_ERR_INVALID_ARG;
  if (!aligned16(q->k_tail) || !aligned16(q->v_tail)) return SFI_ERR_INVALID_ARG;
  if (q->format != SFI_FMT_E4M3 && q->format != SFI_FMT_INT8) return SFI_ERR_UNSUPPORTED;
  return SFI_OK;
}

sfi_status check_index(const sfi_block_index* ix) {
  if (!ix || !ix->bounds || !ix->scale || !ix->page_table) return SFI_ERR_INVALID_ARG;
  if (!aligned16(ix->bounds)) return SFI_ERR_INVALID_ARG;
  return SFI_OK;
}

}  // namespace sfi

using namespace sfi;

extern "C" {

sfi_status sfi_quant_store(const sfi_shape* shape, const sfi_paged_kv* kv, const sfi_quant_kv* qkv,
                           const sfi_block_index* index, int32_t pos_lo, int32_t L, const int32_t* lens,
                           sfi_stream stream) {
  SFI_TRY(check_shape(shape));
  SFI_TRY(check_kv(kv));
  SFI_TRY(check_quant(qkv));
  if (index) SFI_TRY(check_index(index));
  SFI_TRY(check_range(shape, pos_lo, L));
  const int n_pages = (L + kPage - 1) / kPage - pos_lo / kPage;
  if (n_pages <= 0) return SFI_OK;
  QuantArgs a = base_args(*shape, pos_lo, L, lens);
  add_kv(a, *kv);
  add_quant(a, *qkv);
  add_index(a, index);
  const long units = (long)shape->B * n_pages * shape->Hkv * 2;
  const long blocks = (units + 7) / 8;
  if (blocks > 0x7fffffffL) return SFI_ERR_SHAPE;
  const bool e4 = qkv->format == SFI_FMT_E4M3;
  auto k = shape->D == 128 ? (e4 ? store_kernel<128, SFI_FMT_E4M3> : store_kernel<128, SFI_FMT_INT8>)
                           : (e4 ? store_kernel<64, SFI_FMT_E4M3> : store_kernel<64, SFI_FMT_INT8>);
  return launched(launch_k(k, dim3((unsigned)blocks), dim3(256), 0, (cudaStream_t)stream, a, n_pages, units));
}

sfi_status sfi_quant_append(const sfi_shape* shape, const sfi_quant_kv* qkv, const sfi_block_index* index,
                            int32_t L, const int32_t* lens, const sfi_bf16* k_new, const sfi_bf16* v_new,
                            sfi_stream stream) {
  SFI_TRY(check_shape(shape));
  SFI_TRY(check_quant(qkv));
  if (index) SFI_TRY(check_index(index));
  SFI_TRY(check_L(shape, L));
  if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)) return SFI_ERR_INVALID_ARG;
  QuantArgs a = base_args(*shape, 0, L, lens);
  add_quant(a, *qkv);
  add_index(a, index);
  a.k_new = reinterpret_cast<const __nv_bfloat16*>(k_new);
  a.v_new = reinterpret_cast<const __nv_bfloat16*>(v_new);
  const long units = (long)shape->B * shape->Hkv * 2;
  if (units > 0x40000000L) return SFI_ERR_SHAPE;
  const bool e4 = qkv->format == SFI_FMT_E4M3;
  auto k = shape->D == 128 ? (e4 ? append_quant_kernel<128, SFI_FMT_E4M3> : append_quant_kernel<128, SFI_FMT_INT8>)
                           : (e4 ? append_quant_kernel<64, SFI_FMT_E4M3> : append_quant_kernel<64, SFI_FMT_INT8>);
  return launched(
      launch_k(k, dim3((unsigned)((units + 3) / 4)), dim3(128), 0, (cudaStream_t)stream, a, (int)units));
}

sfi_status sfi_quant_load(const sfi_shape* shape, const sfi_quant_kv* qkv, const sfi_paged_kv* kv,
                          int32_t pos_lo, int32_t L, const int32_t* lens, sfi_stream stream) {
  SFI_TRY(check_shape(shape));
  SFI_TRY(check_quant(qkv));
  SFI_TRY(check_kv(kv));
  SFI_TRY(check_range(shape, pos_lo, L));
  const int n_pages = (L + kPage - 1) / kPage - pos_lo / kPage;
  if (n_pages <= 0) return SFI_OK;
  QuantArgs a = base_args(*shape, pos_lo, L, lens);
  add_kv(a, *kv);
  add_quant(a, *qkv);
  const long units = (long)shape->B * n_pages * shape->Hkv * 2;
  const long blocks = (units + 7) / 8;
  if (blocks > 0x7fffffffL) return SFI_ERR_SHAPE;
  const bool e4 = qkv->format == SFI_FMT_E4M3;
  auto k = shape->D == 128 ? (e4 ? load_kernel<128, SFI_FMT_E4M3> : load_kernel<128, SFI_FMT_INT8>)
                           : (e4 ? load_kernel<64, SFI_FMT_E4M3> : load_kernel<64, SFI_FMT_INT8>);
  return launched(launch_k(k, dim3((unsigned)blocks), dim3(256), 0, (cudaStream_t)stream, a, n_pages, units));
}

sfi_status sfi_block_build(const sfi_shape* shape, const sfi_paged_kv* kv, const sfi_block_index* index,
                           int32_t pos_lo, int32_t L, const int32_t* lens, sfi_stream stream) {
  SFI_TRY(check_shape(shape));
  SFI_TRY(check_kv(kv));
  SFI_TRY(check_index(index));
  SFI_TRY(check_range(shape, pos_lo, L));
  const int n_pages = L / kPage - pos_lo / kPage;
  if (n_pages <= 0) return SFI_OK;
  QuantArgs a = base_args(*shape, pos_lo, L, lens);
  add_kv(a, *kv);
  add_index(a, index);
  a.err = index->err;
  const long units = (long)shape->B * n_pages * shape->Hkv;
  const long blocks = (units + 7) / 8;
  if (blocks > 0x7fffffffL) return SFI_ERR_SHAPE;
  auto k = shape->D == 128 ? store_kernel<128, kNoFormat> : store_kernel<64, kNoFormat>;
  return launched(launch_k(k, dim3((unsigned)blocks), dim3(256), 0, (cudaStream_t)stream, a, n_pages, units));
}

sfi_status sfi_quant_poll_error(const sfi_quant_kv* qkv, int32_t* code) {
  if (!qkv || !code) return SFI_ERR_INVALID_ARG;
  sfi_paged_kv kv{};
  kv.err = qkv->err;
  return sfi_poll_error(&kv, code);
}

}  // extern "C"
