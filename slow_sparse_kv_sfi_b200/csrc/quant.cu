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
// Warps of a CTA of the range kernels.  Small CTAs end alone, and their place is
// taken at once: 4 warps took 8K store + load from 94 to 90 us, ragged 32K from
// 421 to 409, against 8.
constexpr unsigned kRangeWarps = 4;

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

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {   // bf16 pairs; NaN stays
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// What a page's codes and bounds go by: its largest magnitude (bf16 bits; 0x7f80
// and above: not finite) and, for keys, each dimension's extremes (this lane's
// 8 values, the same in the lanes of other rows).
struct Extremes {
  uint32_t amax;
  uint32_t hi[4], lo[4];
};
template <int D, bool KEYS>
__device__ __forceinline__ Extremes extremes(const uint4 (&x)[Lay<D>::NI]) {
  using Y = Lay<D>;
  Extremes e;
  uint32_t m = 0;
  if constexpr (KEYS) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      e.hi[j] = e.lo[j] = j == 0 ? x[0].x : j == 1 ? x[0].y : j == 2 ? x[0].z : x[0].w;
#pragma unroll
      for (int i = 1; i < Y::NI; ++i) {
        const uint32_t w = j == 0 ? x[i].x : j == 1 ? x[i].y : j == 2 ? x[i].z : x[i].w;
        e.hi[j] = max2(e.hi[j], w);
        e.lo[j] = min2(e.lo[j], w);
      }
#pragma unroll
      for (int sh = Y::CH; sh < 32; sh <<= 1) {
        e.hi[j] = max2(e.hi[j], __shfl_xor_sync(0xffffffffu, e.hi[j], sh));
        e.lo[j] = min2(e.lo[j], __shfl_xor_sync(0xffffffffu, e.lo[j], sh));
      }
      m = __vmaxu2(m, __vmaxu2(e.hi[j] & 0x7fff7fffu, e.lo[j] & 0x7fff7fffu));
    }
  } else {
#pragma unroll
    for (int i = 0; i < Y::NI; ++i)
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                               __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
  }
  e.amax = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  return e;
}

// Codes and scale of the page in x (this lane's 8 values of NI rows).
template <int D, int FMT>
__device__ __forceinline__ void write_codes(const uint4 (&x)[Lay<D>::NI], uint32_t amax_bits, int lane, uint8_t* codes,
                                            float* scale) {
  using Y = Lay<D>;
  const bool finite = amax_bits < 0x7f80u;
  const float amax = fmaxf(__uint_as_float(amax_bits << 16), kAmaxFloor);
  constexpr float Q = FMT == SFI_FMT_E4M3 ? 448.f : 127.f;
  const float inv = finite ? __fdiv_rn(Q, amax) : 0.f;
  if (lane == 0) *scale = finite ? __fdiv_rn(amax, Q) : __uint_as_float(0x7fc00000u);
  const int row0 = lane / Y::CH, ch = lane % Y::CH;
#pragma unroll
  for (int i = 0; i < Y::NI; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 a = bf2(w[2 * j]), b = bf2(w[2 * j + 1]);
      if constexpr (FMT == SFI_FMT_E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a.x * inv, a.y * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(b.x * inv, b.y * inv), __NV_SATFINITE, __NV_E4M3);
        o[j] = lo | (hi << 16);
      } else {
        // the low byte of 1.5 * 2^23 + y is y rounded to an integer, ties to
        // even (the product is rounded first, as the definition has it)
        const float big = 12582912.f;
        const uint32_t c0 = __float_as_uint(__fadd_rn(__fmul_rn(a.x, inv), big));
        const uint32_t c1 = __float_as_uint(__fadd_rn(__fmul_rn(a.y, inv), big));
        const uint32_t c2 = __float_as_uint(__fadd_rn(__fmul_rn(b.x, inv), big));
        const uint32_t c3 = __float_as_uint(__fadd_rn(__fmul_rn(b.y, inv), big));
        o[j] = __byte_perm(__byte_perm(c0, c1, 0x0040), __byte_perm(c2, c3, 0x0040), 0x5410);
      }
      if (!finite) o[j] = 0u;   // infinity * 0 is not
    }
    *reinterpret_cast<uint2*>(codes + (size_t)(i * Y::RPI + row0) * D + ch * 8) = make_uint2(o[0], o[1]);
  }
}

// Bounds of a page of keys: per dimension the largest and smallest, over the
// page's power-of-two scale, rounded outwards.
template <int D>
__device__ __forceinline__ void write_bounds(const uint4 (&x)[Lay<D>::NI], const Extremes& ex, int lane, int8_t* bounds,
                                             float* scale) {
  using Y = Lay<D>;
  float hi[8], lo[8];
  float amax = __uint_as_float(ex.amax << 16);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = bf2(ex.hi[j]), b = bf2(ex.lo[j]);
    hi[2 * j] = a.x;
    hi[2 * j + 1] = a.y;
    lo[2 * j] = b.x;
    lo[2 * j + 1] = b.y;
  }
  if (ex.amax >= 0x7f80u) {   // not finite: again, with the values that count
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      hi[e] = -INFINITY;
      lo[e] = INFINITY;
    }
#pragma unroll 1
    for (int i = 0; i < Y::NI; ++i) {
      uint4 v = x[0];
#pragma unroll
      for (int k = 1; k < Y::NI; ++k)
        if (k == i) v = x[k];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 a = bf2(w[e / 2]);
        const float u = tame(e % 2 ? a.y : a.x);
        hi[e] = fmaxf(hi[e], u);
        lo[e] = fminf(lo[e], u);
      }
    }
    amax = 0.f;
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
  }
  const int e = unit_exponent(amax);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
  if (lane == 0) *scale = __uint_as_float((uint32_t)(e + 127) << 23);
  if (e > 16) {
    // the quotient of a value far below the scale can underflow to 0 (the
    // smallest bf16 value is 2^-133, the smallest fp32 one 2^-149), which ceil
    // and floor would keep; any value up to the scale gives the same bound
    const float least = __uint_as_float((uint32_t)(e + 127 - 20) << 23);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (hi[k] > 0.f) hi[k] = fmaxf(hi[k], least);
      if (lo[k] < 0.f) lo[k] = fminf(lo[k], -least);
    }
  }
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

// What becomes of a full page in x: codes (FMT != kNoFormat), bounds of its keys.
template <int D, int FMT, bool KEYS>
__device__ __forceinline__ void write_page(const QuantArgs& a, const uint4 (&x)[Lay<D>::NI], int b, int p, int h,
                                           int lane) {
  const Extremes ex = extremes<D, KEYS>(x);
  if constexpr (FMT != kNoFormat) {
    const int dst = page_of(a, a.qpt, b, p, lane, a.err);
    if (dst >= 0) {
      const size_t ph = (size_t)dst * a.Hkv + h;
      write_codes<D, FMT>(x, ex.amax, lane, (KEYS ? a.kq : a.vq) + ph * (kPage * D), (KEYS ? a.ks : a.vs) + ph);
    }
  }
  if constexpr (KEYS) {
    if (a.bounds) {
      const int ip = page_of(a, a.ipt, b, p, lane, a.err_ix);
      if (ip >= 0) {
        const size_t ph = (size_t)ip * a.Hkv + h;
        write_bounds<D>(x, ex, lane, a.bounds + ph * 2 * D, a.bscale + ph);
      }
    }
  }
}

// Work of warp u of sequence b = blockIdx.y in the range kernels: page, KV
// head, K or V (per_page: units of a page).
struct Unit {
  int p, h, v;
};
__device__ __forceinline__ Unit unit_of(uint32_t u, int per_page, int nkv) {
  const uint32_t p = u / (uint32_t)per_page, r = u - p * (uint32_t)per_page;
  return Unit{(int)p, nkv == 2 ? (int)(r >> 1) : (int)r, nkv == 2 ? (int)(r & 1) : 0};
}

// Store: bf16 pages [page_lo, ...) of every sequence -> codes, scales, bounds;
// the page that is not full -> tail.  FMT == kNoFormat: bounds only.
template <int D, int FMT>
__global__ void __launch_bounds__(128) store_kernel(const QuantArgs a, int units) {
  grid_dep_enter_writer();
  using Y = Lay<D>;
  constexpr int nkv = FMT == kNoFormat ? 1 : 2;
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  const uint32_t u = blockIdx.x * kRangeWarps + (threadIdx.x >> 5);
  if (u >= (uint32_t)units) return;
  const Unit w = unit_of(u, a.Hkv * nkv, nkv);
  const int len = seq_len(a.lens, a.L, b, a.err);
  const int p = a.page_lo + w.p;
  const int rows = min(kPage, len - p * kPage);
  if (rows <= 0 || (FMT == kNoFormat && rows < kPage)) return;
  const int src = page_of(a, a.pt, b, p, lane, a.err_kv);
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
    __nv_bfloat16* tail = (w.v ? a.v_tail : a.k_tail) + ((size_t)b * a.Hkv + w.h) * (kPage * D);
#pragma unroll
    for (int i = 0; i < Y::NI; ++i) {
      const int r = i * Y::RPI + row0;
      if (r < rows) *reinterpret_cast<uint4*>(tail + r * D + ch * 8) = x[i];
    }
    return;
  }
  if (w.v) write_page<D, FMT, false>(a, x, b, p, w.h, lane);
  else write_page<D, FMT, true>(a, x, b, p, w.h, lane);
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
    if (v) write_page<D, FMT, false>(a, x, b, p, h, lane);
    else write_page<D, FMT, true>(a, x, b, p, h, lane);
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
__global__ void __launch_bounds__(128) load_kernel(const QuantArgs a, int units) {
  grid_dep_enter_writer();
  using Y = Lay<D>;
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  const uint32_t u = blockIdx.x * kRangeWarps + (threadIdx.x >> 5);
  if (u >= (uint32_t)units) return;
  const Unit w = unit_of(u, a.Hkv * 2, 2);
  const int len = seq_len(a.lens, a.L, b, a.err);
  const int p = a.page_lo + w.p;
  const int rows = min(kPage, len - p * kPage);
  if (rows <= 0) return;
  const int dst = page_of(a, a.pt, b, p, lane, a.err_kv);
  if (dst < 0) return;
  __nv_bfloat16* to = (w.v ? a.v_pool : a.k_pool) + ((size_t)dst * a.Hkv + w.h) * (kPage * D);
  const int row0 = lane / Y::CH, ch = lane % Y::CH;
  if (rows < kPage) {
    const __nv_bfloat16* tail = (w.v ? a.v_tail : a.k_tail) + ((size_t)b * a.Hkv + w.h) * (kPage * D);
#pragma unroll
    for (int i = 0; i < Y::NI; ++i) {
      const int r = i * Y::RPI + row0;
      if (r < rows)
        *reinterpret_cast<uint4*>(to + r * D + ch * 8) = __ldg(reinterpret_cast<const uint4*>(tail + r * D + ch * 8));
    }
    return;
  }
  const int src = page_of(a, a.qpt, b, p, lane, a.err);
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
  const long units = (long)n_pages * shape->Hkv * 2;   // of a sequence
  if (units > 0x7fffff00L || shape->B > 65535) return SFI_ERR_UNSUPPORTED;
  const bool e4 = qkv->format == SFI_FMT_E4M3;
  auto k = shape->D == 128 ? (e4 ? store_kernel<128, SFI_FMT_E4M3> : store_kernel<128, SFI_FMT_INT8>)
                           : (e4 ? store_kernel<64, SFI_FMT_E4M3> : store_kernel<64, SFI_FMT_INT8>);
  return cuda_status(launch_k(k, dim3((unsigned)((units + kRangeWarps - 1) / kRangeWarps), shape->B), dim3(kRangeWarps * 32), 0, (cudaStream_t)stream, a,
                           (int)units));
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
  return cuda_status(
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
  const long units = (long)n_pages * shape->Hkv * 2;   // of a sequence
  if (units > 0x7fffff00L || shape->B > 65535) return SFI_ERR_UNSUPPORTED;
  const bool e4 = qkv->format == SFI_FMT_E4M3;
  auto k = shape->D == 128 ? (e4 ? load_kernel<128, SFI_FMT_E4M3> : load_kernel<128, SFI_FMT_INT8>)
                           : (e4 ? load_kernel<64, SFI_FMT_E4M3> : load_kernel<64, SFI_FMT_INT8>);
  return cuda_status(launch_k(k, dim3((unsigned)((units + kRangeWarps - 1) / kRangeWarps), shape->B), dim3(kRangeWarps * 32), 0, (cudaStream_t)stream, a,
                           (int)units));
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
  const long units = (long)n_pages * shape->Hkv;
  if (units > 0x7fffff00L || shape->B > 65535) return SFI_ERR_UNSUPPORTED;
  auto k = shape->D == 128 ? store_kernel<128, kNoFormat> : store_kernel<64, kNoFormat>;
  return cuda_status(launch_k(k, dim3((unsigned)((units + kRangeWarps - 1) / kRangeWarps), shape->B), dim3(kRangeWarps * 32), 0, (cudaStream_t)stream, a,
                           (int)units));
}

sfi_status sfi_quant_poll_error(const sfi_quant_kv* qkv, int32_t* code) {
  if (!qkv || !code) return SFI_ERR_INVALID_ARG;
  sfi_paged_kv kv{};
  kv.err = qkv->err;
  return sfi_poll_error(&kv, code);
}

}  // extern "C"
