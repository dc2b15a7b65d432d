// Block selection: a score for every page ("block" of 16 tokens) of a
// (sequence, KV head) from the int8 bounds of its keys, and the K best.
//
//   u_j = max_h e_h * scale_j * sum_d max(q^_hd hi_jd, q^_hd lo_jd)
//
// Since hi >= lo, the maximum is q^+ . hi + q^- . lo with q^+ = max(q^, 0) and
// q^- = min(q^, 0): one int8 dot product of length 2 D with the page's bounds
// row [hi | lo], for all heads of the group at once on the int8 tensor path
// (m16n8k32: 16 pages x 8 heads).  |sum| <= 127 * 127 * D < 2^24 and the
// scales are powers of two, so u is exact in fp32 and does not depend on the
// order of the sum.
//
// Bound by reading 2 D bytes per (page, KV head).  A thread loads the bytes of
// its fragment straight from global memory: the order of d inside the dot
// product is free as long as q uses the same one, so thread t of a quad takes
// the 16-byte chunks t, t + 4, ... of its two rows.
#include "common.cuh"
#include "internal.h"

namespace sfi {
namespace {

constexpr int kScoreWarps = 8;

struct BlockScoreArgs {
  int B, Hq, Hkv, G, L, num_pages, max_pages, nb;
  int n_sink, n_recent;
  const int32_t* lens;
  const __nv_bfloat16* q;
  const int8_t* bounds;
  const float* scale;
  const int32_t* pt;
  float* scores;
  int64_t ld;
  int* err;
};

__device__ __forceinline__ void mma_s8_16832(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float tame(float x) {
  const float big = __uint_as_float(0x7f7f0000u);
  return x != x ? 0.f : fminf(fmaxf(x, -big), big);
}

template <int D, int NT>
__global__ void __launch_bounds__(kScoreWarps * 32) block_score_kernel(const BlockScoreArgs a) {
  grid_dep_enter();
  constexpr int KC = 2 * D / 64;   // 16-byte chunks per thread and row
  __shared__ __align__(16) int8_t qc[NT * 8][2 * D];
  __shared__ float qe[NT * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.y, b = bh / a.Hkv, h = bh - b * a.Hkv;

  // the group's query codes, split by sign
  for (int n = warp; n < NT * 8; n += kScoreWarps) {
    constexpr int E = D / 32;
    float x[E];
    float am = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] = n < a.G ? tame(__bfloat162float(a.q[((size_t)b * a.Hq + h * a.G + n) * D + lane * E + e])) : 0.f;
      am = fmaxf(am, fabsf(x[e]));
    }
#pragma unroll
    for (int sh = 16; sh >= 1; sh >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, sh));
    const int ex = unit_exponent(am);
    const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = __float2int_rn(x[e] * inv);
      qc[n][lane * E + e] = (int8_t)max(c, 0);
      qc[n][D + lane * E + e] = (int8_t)min(c, 0);
    }
    if (lane == 0) qe[n] = __uint_as_float((uint32_t)(ex + 127) << 23);
  }
  __syncthreads();

  const int len = seq_len(a.lens, a.L, b, a.err);
  const int r0 = lane >> 2, t = lane & 3;
  uint32_t qb[NT][KC][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < KC; ++j)
#pragma unroll
      for (int w = 0; w < 4; ++w)
        qb[nt][j][w] = *reinterpret_cast<const uint32_t*>(&qc[nt * 8 + r0][(t + 4 * j) * 16 + 4 * w]);

  const int n_tiles = (a.nb + 15) / 16;
  for (int tile = blockIdx.x * kScoreWarps + warp; tile < n_tiles; tile += gridDim.x * kScoreWarps) {
    uint4 x[2][KC];
    float sc[2];
    float forced[2];   // the score where it does not come from the bounds, else NaN
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int j = tile * 16 + r0 + 8 * r;
      sc[r] = 0.f;
      forced[r] = __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int c = 0; c < KC; ++c) x[r][c] = make_uint4(0, 0, 0, 0);
      if (j * kPage >= len) {
        forced[r] = -INFINITY;
      } else if (j * kPage < a.n_sink || (j + 1) * kPage > len - a.n_recent) {
        forced[r] = INFINITY;
      } else {
        const int page = __ldg(a.pt + (size_t)b * a.max_pages + j);
        if ((unsigned)page >= (unsigned)a.num_pages) {
          latch_error(a.err, SFI_ERR_DEVICE_CHECK, kSiteBlockPage);
          forced[r] = -INFINITY;
        } else {
          const size_t ph = (size_t)page * a.Hkv + h;
          const uint4* row = reinterpret_cast<const uint4*>(a.bounds + ph * 2 * D);
#pragma unroll
          for (int c = 0; c < KC; ++c) x[r][c] = __ldg(row + t + 4 * c);
          sc[r] = __ldg(a.scale + ph);
        }
      }
    }
    float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      int d[4] = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint32_t a0[4] = {x[0][c].x, x[1][c].x, x[0][c].y, x[1][c].y};
        const uint32_t a1[4] = {x[0][c].z, x[1][c].z, x[0][c].w, x[1][c].w};
        mma_s8_16832(d, a0, qb[nt][c][0], qb[nt][c][1]);
        mma_s8_16832(d, a1, qb[nt][c][2], qb[nt][c][3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = nt * 8 + 2 * t + (i & 1);
        if (n < a.G) best[i >> 1] = fmaxf(best[i >> 1], (float)d[i] * qe[n]);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
      best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
      const int j = tile * 16 + r0 + 8 * r;
      if (t == r && j < a.nb) {
        const float big = __uint_as_float(0x7f7fffffu);
        const float u = fminf(fmaxf(best[r] * sc[r], -big), big);
        a.scores[(size_t)bh * a.ld + j] = forced[r] == forced[r] ? forced[r] : u;
      }
    }
  }
}

#define SFI_TRY(x)               \
  do {                           \
    sfi_status _r = (x);         \
    if (_r != SFI_OK) return _r; \
  } while (0)

}  // namespace

BlockWs block_ws(const sfi_shape& s) {
  BlockWs w{};
  const long long BH = (long long)s.B * s.Hkv;
  const int G = s.Hq / s.Hkv;
  size_t off = 0;
  w.score_off = off;
  off += align_up((size_t)BH * (((size_t)s.max_pages + 3) / 4 * 4) * sizeof(float), 256);
  const size_t items = 2 * (size_t)page_attn_ctas(BH * s.max_pages, 4);
  w.part_off = off;
  off += align_up(items * G * s.D * sizeof(float), 256);
  w.ml_off = off;
  off += align_up(items * G * 2 * sizeof(float), 256);
  w.total = off;
  return w;
}

}  // namespace sfi

using namespace sfi;

extern "C" {

sfi_status sfi_block_workspace_size(const sfi_shape* shape, size_t* bytes) {
  SFI_TRY(check_shape(shape));
  if (!bytes) return SFI_ERR_INVALID_ARG;
  *bytes = block_ws(*shape).total;
  return SFI_OK;
}

sfi_status sfi_block_select(const sfi_shape* shape, const sfi_block_index* index, int32_t L, const int32_t* lens,
                            const sfi_bf16* q, int32_t n_sink, int32_t n_recent, int32_t K, int32_t* sel,
                            int32_t sel_ld, void* ws, size_t ws_bytes, sfi_stream stream) {
  SFI_TRY(check_shape(shape));
  SFI_TRY(check_index(index));
  SFI_TRY(check_L(shape, L));
  if (!q || !aligned16(q) || !sel) return SFI_ERR_INVALID_ARG;
  if (n_sink < 0 || n_recent < 1) return SFI_ERR_SHAPE;
  const int nb = (L + kPage - 1) / kPage;
  const long always = ((long)n_sink + kPage - 1) / kPage + ((long)n_recent + kPage - 1) / kPage + 1;
  if (K < 1 || K > nb || K < (always < nb ? always : nb) || sel_ld < K) return SFI_ERR_SHAPE;
  if (nb > topk_max_n() || (long)shape->B * shape->Hkv > 65535) return SFI_ERR_UNSUPPORTED;
  const BlockWs w = block_ws(*shape);
  if (!ws || !aligned16(ws) || ws_bytes < w.total) return SFI_ERR_WORKSPACE;
  const int BH = shape->B * shape->Hkv;
  BlockScoreArgs a{};
  a.B = shape->B;
  a.Hq = shape->Hq;
  a.Hkv = shape->Hkv;
  a.G = shape->Hq / shape->Hkv;
  a.L = L;
  a.num_pages = shape->num_pages;
  a.max_pages = shape->max_pages;
  a.nb = nb;
  a.n_sink = n_sink;
  a.n_recent = n_recent;
  a.lens = lens;
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.bounds = index->bounds;
  a.scale = index->scale;
  a.pt = index->page_table;
  a.scores = reinterpret_cast<float*>(static_cast<char*>(ws) + w.score_off);
  a.ld = (nb + 3) / 4 * 4;
  a.err = index->err;
  cudaStream_t st = (cudaStream_t)stream;
  // one tile of 16 pages per warp until the grid fills the GPU about twice
  // (256-thread CTAs, several per SM); longer rows loop
  const int tiles = (nb + 15) / 16;
  int gx = (tiles + kScoreWarps - 1) / kScoreWarps;
  const int cap = (num_sms() * 8 + BH - 1) / BH;
  if (gx > cap) gx = cap;
  const dim3 grid(gx, BH);
  const bool wide = a.G > 8;
  auto k = shape->D == 128 ? (wide ? block_score_kernel<128, 2> : block_score_kernel<128, 1>)
                           : (wide ? block_score_kernel<64, 2> : block_score_kernel<64, 1>);
  if (launch_k(k, grid, dim3(kScoreWarps * 32), 0, st, a) != cudaSuccess) {
    cudaGetLastError();
    return SFI_ERR_CUDA;
  }
  return run_topk(BH, nb, a.scores, a.ld, K, 0, sel, sel_ld, nullptr, 0, st);
}

}  // extern "C"
