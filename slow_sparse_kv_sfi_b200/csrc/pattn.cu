// Decode attention over pages: all pages of an 8-bit cache, or listed pages of
// an 8-bit or a bf16 cache.
//
//   z_j = q . k_j / sqrt(D),  out = sum_j softmax(z)_j v_j
//
// Work.  The pages (or list entries) of one (sequence, KV head) are cut into
// chunks, one CTA each; warp w of the CTA takes tiles w, w + W, ... of its
// chunk, a tile being one page: 16 rows of K and of V.  Each warp runs its own
// online softmax; the CTA merges its warps in shared memory, and a second
// kernel merges the chunks.
//
// Bound by reading the cache, so the layout serves the loads.  Every warp
// streams its tiles through its own ring of stages with 16-byte asynchronous
// copies, and each thread copies exactly the bytes its own matrix fragments
// need: no barrier, no swizzle, no bank conflict, and no wait that another
// warp has to end.  That works because the order of a contraction is free:
//   S^T[16 tok x 8 heads] = K[16 x D] . Q^T[D x 8]: thread (g, t) of the
//     fragment layout (g = lane / 4, t = lane % 4) holds rows g, g + 8 and any
//     D / 4 of the columns, as long as Q is laid out alike: the 16-byte chunks
//     t, t + 4, ... of the row;
//   O^T[D x 8 heads] += V^T[D x 16] . P^T[16 x 8]: it holds tokens 2t, 2t + 1,
//     2t + 8, 2t + 9 and a run of D / 8 columns of each; two tokens' bytes are
//     interleaved into the 16-bit pairs that the fragment wants.
// 8-bit codes become bf16 in registers, exactly (int8 and e4m3 both fit); the
// key scale multiplies the logits, the value scale the probabilities.
// P is split into bf16 hi + lo, which keeps about 16 bits of it.
// The running maximum moves only when a logit exceeds it by 6 (P up to 64, far
// from overflow), so most tiles need no rescaling and no reduction.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace sfi {
namespace {

constexpr int kBf16 = 2;            // FMT: SFI_FMT_E4M3, SFI_FMT_INT8 or this
constexpr float kSlack = 6.f;       // log2 of the largest P

struct PageAttnArgs {
  int B, Hq, Hkv, G, L, num_pages, max_pages;
  const int32_t* lens;
  const int32_t* pt;
  const __nv_bfloat16* q;
  const uint8_t* k;                 // pools (bytes)
  const uint8_t* v;
  const float* ks;
  const float* vs;
  const __nv_bfloat16* k_tail;
  const __nv_bfloat16* v_tail;
  const int32_t* sel;               // LIST
  int64_t sel_ld;
  int K;
  int chunk;                        // tiles per chunk
  int n_chunks;
  float scale_log2;                 // log2(e) / sqrt(D)
  float* out;
  float* lse;
  float* part;                      // [item][G][D]
  float* ml;                        // [item][G][2]
  int* err;
};

template <int D, int FMT, int NT>
struct Cfg {
  static constexpr int kEl = FMT == kBf16 ? 2 : 1;
  static constexpr int kRow = D * kEl;                  // bytes of a row
  static constexpr int KJ = kRow / 64;                  // 16-byte chunks of a K row per thread
  static constexpr int kVB = kRow / 8;                  // bytes of a V row per thread: 8, 16 or 32
  static constexpr int VC = kVB >= 16 ? kVB / 16 : 1;   // pieces of them
  static constexpr int VP = kVB >= 16 ? 16 : 8;         // bytes of a piece
  static constexpr int kKBytes = 16 * kRow;             // of a stage, K and V alike
  static constexpr int kStage = 2 * kKBytes;
  // Warps and stages: about 96 KB of copies in flight per SM at two CTAs (one
  // for G > 8, whose accumulators need twice the registers).
  static constexpr int W = FMT == kBf16 ? 4 : 8;
  static constexpr int kCtas = NT == 1 ? 2 : 1;
  static constexpr int S = D == 64 ? 4 : 3;
  static constexpr int kRing = W * S * kStage;
  static constexpr int kMerge = W * NT * 8 * (D + 8) * 4 + W * NT * 8 * 2 * 4;
  static constexpr int kMeta = W * S * 16;
  static constexpr int kSmem = (kRing > kMerge ? kRing : kMerge) + kMeta;
};

struct Meta {       // of a stage
  int page;         // >= 0; -1: nothing; -2: the tail
  int rows;         // valid rows
  float ks, vs;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ uint2 lds8(const uint8_t* p) { return *reinterpret_cast<const uint2*>(p); }

// Bytes 0, 2 of v -> ev and bytes 1, 3 -> od, as bf16 pairs.
//  int8: x = low7 - 128 s (s the sign bit); 0x4300 | low7 is 128 + low7 and
//        0x4300 | 0x80 s is 128 + 128 s in bf16, so their difference is x.
//  e4m3: sign, exponent and mantissa bits moved to their bf16 places are the
//        value times 2^(7 - 127), subnormals included; times 2^120.
template <int FMT>
__device__ __forceinline__ void to_bf16(uint32_t v, uint32_t& ev, uint32_t& od) {
  if constexpr (FMT == SFI_FMT_INT8) {
    const uint32_t o = v >> 8;
    const uint32_t a = (v & 0x007f007fu) | 0x43004300u, b = (v & 0x00800080u) | 0x43004300u;
    const uint32_t c = (o & 0x007f007fu) | 0x43004300u, d = (o & 0x00800080u) | 0x43004300u;
    const __nv_bfloat162 e = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    const __nv_bfloat162 f = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c), *reinterpret_cast<const __nv_bfloat162*>(&d));
    ev = *reinterpret_cast<const uint32_t*>(&e);
    od = *reinterpret_cast<const uint32_t*>(&f);
  } else {
    const uint32_t a = ((v << 4) & 0x07f007f0u) | ((v << 8) & 0x80008000u);
    const uint32_t b = ((v >> 4) & 0x07f007f0u) | (v & 0x80008000u);
    const uint32_t m = 0x7b807b80u;   // 2^120, twice
    const __nv_bfloat162 k = *reinterpret_cast<const __nv_bfloat162*>(&m);
    const __nv_bfloat162 e = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), k);
    const __nv_bfloat162 f = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b), k);
    ev = *reinterpret_cast<const uint32_t*>(&e);
    od = *reinterpret_cast<const uint32_t*>(&f);
  }
}

__device__ __forceinline__ uint32_t word(const uint4& x, int w) { return w == 0 ? x.x : w == 1 ? x.y : w == 2 ? x.z : x.w; }

// The state of one warp: running maximum (log2 units) and this thread's share
// of the sum for heads 2t, 2t + 1 of each head tile, and O^T.
template <int D, int NT>
struct State {
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];
};

// One tile from its fragments: kf(step, a[4]) and vf(step, a[4]) fill the A
// operands of S^T and O^T.  rows: valid rows of the tile.
template <int D, int NT, class KF, class VF>
__device__ __forceinline__ void tile_math(State<D, NT>& st, const uint32_t (&qb)[NT][D / 16][2], float zf, float vs,
                                          int rows, int lane, KF kf, VF vf) {
  float s[NT][4], s2[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[nt][i] = s2[nt][i] = 0.f;
#pragma unroll
  for (int k = 0; k < D / 16; k += 2) {
    uint32_t a[4], b[4];
    kf(k, a);
    kf(k + 1, b);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mma_bf16_16816(s[nt], a, qb[nt][k][0], qb[nt][k][1]);
      mma_bf16_16816(s2[nt], b, qb[nt][k + 1][0], qb[nt][k + 1][1]);
    }
  }
  bool grow = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[nt][i] = (s[nt][i] + s2[nt][i]) * zf;
      if (rows < kPage && (lane >> 2) + 8 * (i >> 1) >= rows) s[nt][i] = -INFINITY;
      grow |= s[nt][i] > st.m[nt][i & 1] + kSlack;
    }
  if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = fmaxf(s[nt][j], s[nt][j + 2]);
#pragma unroll
        for (int sh = 4; sh <= 16; sh <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, sh));
        const float mn = fmaxf(st.m[nt][j], x);
        const float al = mn == -INFINITY ? 1.f : fast_exp2(st.m[nt][j] - mn);
        st.m[nt][j] = mn;
        st.l[nt][j] *= al;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          st.o[nt][k][j] *= al;
          st.o[nt][k][j + 2] *= al;
        }
      }
  }
  uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float p[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float m = st.m[nt][j] == -INFINITY ? 0.f : st.m[nt][j];
        p[j] = fast_exp2(s[nt][2 * r + j] - m);
        st.l[nt][j] += p[j];
        p[j] *= vs;
      }
      const uint32_t h = pack_bf16x2(p[0], p[1]);
      const float2 f = unpack_bf16x2(h);
      hi[nt][r] = movmatrix_trans(h);
      lo[nt][r] = movmatrix_trans(pack_bf16x2(p[0] - f.x, p[1] - f.y));
    }
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    uint32_t a[4];
    vf(k, a);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mma_bf16_16816(st.o[nt][k], a, hi[nt][0], hi[nt][1]);
      mma_bf16_16816(st.o[nt][k], a, lo[nt][0], lo[nt][1]);
    }
  }
}

template <int D, int FMT, int NT, bool LIST>
__global__ void __launch_bounds__(Cfg<D, FMT, NT>::W * 32, Cfg<D, FMT, NT>::kCtas)
    page_attn_kernel(const __grid_constant__ PageAttnArgs a) {
  using C = Cfg<D, FMT, NT>;
  constexpr int W = C::W, S = C::S, KJ = C::KJ, VC = C::VC, VP = C::VP;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int bh = blockIdx.y, b = bh / a.Hkv, h = bh - b * a.Hkv;
  grid_dep_wait();
  if (a.n_chunks > 1) grid_dep_launch();

  const int len = seq_len(a.lens, a.L, b, a.err);
  const int blocks = (len + kPage - 1) / kPage;
  const int T = LIST ? a.K : blocks;
  const int t0 = blockIdx.x * a.chunk, t1 = min(T, t0 + a.chunk);
  if (!LIST && t0 >= T && a.n_chunks > 1) return;   // the merge kernel counts chunks alike

  // queries of the group: B operands of S^T, in the column order of the K
  // fragments (zero for heads past G)
  uint32_t qb[NT][D / 16][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int n = nt * 8 + g;
    const __nv_bfloat16* q = a.q + ((size_t)b * a.Hq + h * a.G + (n < a.G ? n : 0)) * D;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const int d = FMT == kBf16 ? (t + 4 * (k / 2)) * 8 + (k % 2) * 4 : (t + 4 * (k / 4)) * 16 + (k % 4) * 4;
      uint2 x = __ldg(reinterpret_cast<const uint2*>(q + d));
      if (n >= a.G) x = make_uint2(0, 0);
      qb[nt][k][0] = FMT == kBf16 ? x.x : __byte_perm(x.x, x.y, 0x5410);
      qb[nt][k][1] = FMT == kBf16 ? x.y : __byte_perm(x.x, x.y, 0x7632);
    }
  }

  uint8_t* ring = smem + (size_t)warp * S * C::kStage;
  const uint32_t ring_u = smem_u32(ring) + lane * 16;
  Meta* meta = reinterpret_cast<Meta*>(smem + (C::kSmem - C::kMeta)) + warp * S;

  // Tiles of this warp: t0 + warp + W * i, i < n.  Lane l looks up tile
  // i0 + l of a batch of 32: block, page and scales.
  const int n = t1 - t0 > warp ? (t1 - t0 - warp + W - 1) / W : 0;
  Meta mine{-1, 0, 0.f, 0.f};
  auto look_up = [&](int i0) {
    mine = Meta{-1, 0, 0.f, 0.f};
    const int i = i0 + lane;
    if (i >= n) return;
    const int tile = t0 + warp + W * i;
    const int blk = LIST ? __ldg(a.sel + (size_t)bh * a.sel_ld + tile) : tile;
    if ((unsigned)blk >= (unsigned)blocks) return;
    mine.rows = min(kPage, len - blk * kPage);
    if (FMT != kBf16 && mine.rows < kPage) {
      mine.page = -2;
      return;
    }
    const int page = __ldg(a.pt + (size_t)b * a.max_pages + blk);
    if ((unsigned)page >= (unsigned)a.num_pages) {
      latch_error(a.err, SFI_ERR_DEVICE_CHECK, kSitePageAttn);
      return;
    }
    mine.page = page;
    if (FMT != kBf16) {
      mine.ks = __ldg(a.ks + (size_t)page * a.Hkv + h);
      mine.vs = __ldg(a.vs + (size_t)page * a.Hkv + h);
    }
  };

  // copies of tile i into stage i % S
  auto issue = [&](int i) {
    if (i < n) {
      if ((i & 31) == 0) look_up(i);
      const int src = i & 31;
      if (lane == src) meta[i % S] = mine;
      const int page = __shfl_sync(0xffffffffu, mine.page, src);
      if (page >= 0) {
        const size_t off = ((size_t)page * a.Hkv + h) * C::kKBytes;
        const uint8_t* kp = a.k + off + g * C::kRow + t * 16;
        const uint8_t* vp = a.v + off + 2 * t * C::kRow + g * VP;
        const uint32_t sk = ring_u + (i % S) * C::kStage, sv = sk + C::kKBytes;
        if constexpr (FMT == kBf16) {
          const int rows = __shfl_sync(0xffffffffu, mine.rows, src);
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < KJ; ++j)
              cp_async16_zfill(sk + (r * KJ + j) * 512, kp + r * 8 * C::kRow + j * 64, g + 8 * r < rows ? 16 : 0);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int tok = (x & 1) + 8 * (x >> 1);
#pragma unroll
            for (int c = 0; c < VC; ++c)
              cp_async16_zfill(sv + (x * VC + c) * 512, vp + tok * C::kRow + c * 128, 2 * t + tok < rows ? 16 : 0);
          }
        } else {
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < KJ; ++j)
              cp_async16(sk + (r * KJ + j) * 512, kp + r * 8 * C::kRow + j * 64);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int tok = (x & 1) + 8 * (x >> 1);
            if constexpr (VP == 16) cp_async16(sv + x * 512, vp + tok * C::kRow);
            else cp_async8(sv - lane * 8 + x * 256, vp + tok * C::kRow);
          }
        }
      }
    }
    cp_commit();
  };

  State<D, NT> st;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      st.m[nt][j] = -INFINITY;
      st.l[nt][j] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[nt][k][i] = 0.f;
  }

#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);
  for (int i = 0; i < n; ++i) {
    __syncwarp();   // every lane has read stage (i - 1) % S's description
    issue(i + S - 1);
    cp_wait<S - 1>();
    __syncwarp();
    const Meta mt = meta[i % S];
    const uint8_t* sk = ring + (i % S) * C::kStage + lane * 16;
    const uint8_t* sv = sk + C::kKBytes;
    if (mt.page >= 0) {
      if constexpr (FMT == kBf16) {
        tile_math<D, NT>(
            st, qb, a.scale_log2, 1.f, mt.rows, lane,
            [&](int k, uint32_t (&f)[4]) {
              const uint4 x = lds16(sk + (k / 2) * 512), y = lds16(sk + (KJ + k / 2) * 512);
              const int w = (k % 2) * 2;
              f[0] = word(x, w);
              f[1] = word(y, w);
              f[2] = word(x, w + 1);
              f[3] = word(y, w + 1);
            },
            [&](int k, uint32_t (&f)[4]) {
              const int c = k / 4, w = k % 4;
              const uint32_t x0 = word(lds16(sv + c * 512), w), x1 = word(lds16(sv + (VC + c) * 512), w);
              const uint32_t x2 = word(lds16(sv + (2 * VC + c) * 512), w), x3 = word(lds16(sv + (3 * VC + c) * 512), w);
              f[0] = __byte_perm(x0, x1, 0x5410);
              f[1] = __byte_perm(x0, x1, 0x7632);
              f[2] = __byte_perm(x2, x3, 0x5410);
              f[3] = __byte_perm(x2, x3, 0x7632);
            });
      } else {
        tile_math<D, NT>(
            st, qb, a.scale_log2 * mt.ks, mt.vs, kPage, lane,
            [&](int k, uint32_t (&f)[4]) {
              to_bf16<FMT>(word(lds16(sk + (k / 4) * 512), k % 4), f[0], f[2]);
              to_bf16<FMT>(word(lds16(sk + (KJ + k / 4) * 512), k % 4), f[1], f[3]);
            },
            [&](int k, uint32_t (&f)[4]) {
              uint32_t x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if constexpr (VP == 16) {
                  x[i] = word(lds16(sv + i * 512), k / 2);
                } else {
                  const uint2 y = lds8(sv - lane * 8 + i * 256);
                  x[i] = k / 2 == 0 ? y.x : y.y;
                }
              }
              const uint32_t sel = k % 2 ? 0x7632 : 0x5410;
              to_bf16<FMT>(__byte_perm(x[0], x[1], sel), f[0], f[1]);
              to_bf16<FMT>(__byte_perm(x[2], x[3], sel), f[2], f[3]);
            });
      }
    } else if (FMT != kBf16 && mt.page == -2) {
      // the bf16 rows of the page that is not full, straight from memory, in
      // the column orders of the 8-bit fragments
      const __nv_bfloat16* kt = a.k_tail + (size_t)bh * (kPage * D);
      const __nv_bfloat16* vt = a.v_tail + (size_t)bh * (kPage * D);
      const int rows = mt.rows;
      tile_math<D, NT>(
          st, qb, a.scale_log2, 1.f, rows, lane,
          [&](int k, uint32_t (&f)[4]) {
            const int d = (t + 4 * (k / 4)) * 16 + (k % 4) * 4;
            uint2 x = make_uint2(0, 0), y = make_uint2(0, 0);
            if (g < rows) x = __ldg(reinterpret_cast<const uint2*>(kt + g * D + d));
            if (g + 8 < rows) y = __ldg(reinterpret_cast<const uint2*>(kt + (g + 8) * D + d));
            f[0] = __byte_perm(x.x, x.y, 0x5410);
            f[1] = __byte_perm(y.x, y.y, 0x5410);
            f[2] = __byte_perm(x.x, x.y, 0x7632);
            f[3] = __byte_perm(y.x, y.y, 0x7632);
          },
          [&](int k, uint32_t (&f)[4]) {
            const int d = g * (D / 8) + 2 * k;
            uint32_t x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tok = 2 * t + (i & 1) + 8 * (i >> 1);
              x[i] = tok < rows ? __ldg(reinterpret_cast<const uint32_t*>(vt + tok * D + d)) : 0u;
            }
            f[0] = __byte_perm(x[0], x[1], 0x5410);
            f[1] = __byte_perm(x[0], x[1], 0x7632);
            f[2] = __byte_perm(x[2], x[3], 0x5410);
            f[3] = __byte_perm(x[2], x[3], 0x7632);
          });
    }
  }
  cp_wait<0>();

  // Merge of the CTA's warps: O of each head, row of D floats padded by 8,
  // then (m, l) of each head.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int sh = 4; sh <= 16; sh <<= 1) st.l[nt][j] += __shfl_xor_sync(0xffffffffu, st.l[nt][j], sh);
  __syncthreads();   // every warp is done with its ring
  constexpr int kLd = D + 8;
  float* so = reinterpret_cast<float*>(smem);
  float* sml = so + W * NT * 8 * kLd;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      int d;
      if (FMT == kBf16) d = (k / 4) * 64 + g * 8 + (k % 4) * 2;
      else d = g * (D / 8) + 2 * k;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<float2*>(so + (size_t)(warp * NT * 8 + nt * 8 + 2 * t + j) * kLd + d) =
            make_float2(st.o[nt][k][j], st.o[nt][k][j + 2]);
    }
  if (g == 0) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<float2*>(sml + (warp * NT * 8 + nt * 8 + 2 * t + j) * 2) =
            make_float2(st.m[nt][j], st.l[nt][j]);
  }
  __syncthreads();
  const int item = bh * a.n_chunks + blockIdx.x;
  for (int e = threadIdx.x; e < a.G * D; e += W * 32) {
    const int n_ = e / D, d = e - n_ * D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, sml[(w * NT * 8 + n_) * 2]);
    const float ref = M == -INFINITY ? 0.f : M;
    float l = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = fast_exp2(sml[(w * NT * 8 + n_) * 2] - ref);
      l += f * sml[(w * NT * 8 + n_) * 2 + 1];
      o += f * so[(size_t)(w * NT * 8 + n_) * kLd + d];
    }
    if (a.n_chunks == 1) {
      const size_t row = (size_t)b * a.Hq + h * a.G + n_;
      a.out[row * D + d] = l == 0.f ? 0.f : o / l;
      if (d == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (M + fast_log2(l)) * kLn2;
    } else {
      a.part[((size_t)item * a.G + n_) * D + d] = o;
      if (d == 0) *reinterpret_cast<float2*>(a.ml + ((size_t)item * a.G + n_) * 2) = make_float2(M, l);
    }
  }
}

// Merge of the chunks of one (sequence, query head): D threads per group of
// chunks, four groups.
template <int D>
__global__ void __launch_bounds__(4 * D) page_merge_kernel(const __grid_constant__ PageAttnArgs a, int list) {
  grid_dep_wait();
  __shared__ float so[4][D], sl[4], sm[4];
  const int row = blockIdx.x, b = row / a.Hq, hq = row - b * a.Hq;
  const int h = hq / a.G, n_ = hq - h * a.G;
  const int grp = threadIdx.x / D, d = threadIdx.x % D;
  const int len = seq_len(a.lens, a.L, b, nullptr);
  const int T = list ? a.K : (len + kPage - 1) / kPage;
  const int nc = (T + a.chunk - 1) / a.chunk;
  const size_t first = (size_t)(b * a.Hkv + h) * a.n_chunks;
  float M = -INFINITY, l = 0.f, o = 0.f;
  for (int c = grp; c < nc; c += 4) {
    const size_t r = (first + c) * a.G + n_;
    const float2 ml = __ldg(reinterpret_cast<const float2*>(a.ml + r * 2));
    const float x = __ldg(a.part + r * D + d);
    const float mn = fmaxf(M, ml.x);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float f0 = fast_exp2(M - ref), f1 = fast_exp2(ml.x - ref);
    l = l * f0 + ml.y * f1;
    o = o * f0 + x * f1;
    M = mn;
  }
  so[grp][d] = o;
  if (d == 0) {
    sl[grp] = l;
    sm[grp] = M;
  }
  __syncthreads();
  if (grp != 0) return;
  M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  const float ref = M == -INFINITY ? 0.f : M;
  l = o = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = fast_exp2(sm[i] - ref);
    l += f * sl[i];
    o += f * so[i][d];
  }
  a.out[(size_t)row * D + d] = l == 0.f ? 0.f : o / l;
  if (d == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (M + fast_log2(l)) * kLn2;
}

#define SFI_TRY(x)               \
  do {                           \
    sfi_status _r = (x);         \
    if (_r != SFI_OK) return _r; \
  } while (0)

sfi_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return SFI_OK;
  cudaGetLastError();
  return SFI_ERR_CUDA;
}

template <int D, int FMT, int NT, bool LIST>
sfi_status launch(const PageAttnArgs& a, cudaStream_t st) {
  using C = Cfg<D, FMT, NT>;
  auto k = page_attn_kernel<D, FMT, NT, LIST>;
  static DeviceOnce once;
  if (!once.done()) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (!once.mark(e)) return cuda_status(e);
  }
  const sfi_status r = cuda_status(launch_k(k, dim3(a.n_chunks, a.B * a.Hkv), dim3(C::W * 32), C::kSmem, st, a));
  if (r != SFI_OK || a.n_chunks == 1) return r;
  return cuda_status(launch_k(page_merge_kernel<D>, dim3(a.B * a.Hq), dim3(4 * D), 0, st, a, LIST ? 1 : 0));
}

template <int FMT, bool LIST>
sfi_status launch_any(int D, const PageAttnArgs& a, cudaStream_t st) {
  if (D == 128) return a.G > 8 ? launch<128, FMT, 2, LIST>(a, st) : launch<128, FMT, 1, LIST>(a, st);
  return a.G > 8 ? launch<64, FMT, 2, LIST>(a, st) : launch<64, FMT, 1, LIST>(a, st);
}

// Shared by the three entry points: kv (bf16) or q8 (8-bit) is the cache.
sfi_status run(const sfi_shape* shape, const sfi_paged_kv* kv, const sfi_quant_kv* q8, int32_t L, const int32_t* lens,
               const sfi_bf16* q, const int32_t* sel, int32_t sel_ld, int32_t K, bool list, float* out, float* lse,
               void* ws, size_t ws_bytes, sfi_stream stream) {
  SFI_TRY(check_shape(shape));
  SFI_TRY(q8 ? check_quant(q8) : check_kv(kv));
  SFI_TRY(check_L(shape, L));
  if (!q || !aligned16(q) || !out) return SFI_ERR_INVALID_ARG;
  if (list) {
    if (!sel) return SFI_ERR_INVALID_ARG;
    if (K < 1 || sel_ld < K) return SFI_ERR_SHAPE;
    if (K > shape->max_pages) return SFI_ERR_SHAPE;
  }
  const long BHl = (long)shape->B * shape->Hkv;
  if (BHl > 65535) return SFI_ERR_UNSUPPORTED;
  const BlockWs w = block_ws(*shape);
  if (!ws || !aligned16(ws) || ws_bytes < w.total) return SFI_ERR_WORKSPACE;
  const int BH = (int)BHl;
  PageAttnArgs a{};
  a.B = shape->B;
  a.Hq = shape->Hq;
  a.Hkv = shape->Hkv;
  a.G = shape->Hq / shape->Hkv;
  a.L = L;
  a.num_pages = shape->num_pages;
  a.max_pages = shape->max_pages;
  a.lens = lens;
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  if (q8) {
    a.pt = q8->page_table;
    a.k = q8->k_pool;
    a.v = q8->v_pool;
    a.ks = q8->k_scale;
    a.vs = q8->v_scale;
    a.k_tail = reinterpret_cast<const __nv_bfloat16*>(q8->k_tail);
    a.v_tail = reinterpret_cast<const __nv_bfloat16*>(q8->v_tail);
    a.err = q8->err;
  } else {
    a.pt = kv->page_table;
    a.k = reinterpret_cast<const uint8_t*>(kv->k_pool);
    a.v = reinterpret_cast<const uint8_t*>(kv->v_pool);
    a.err = kv->err;
  }
  a.sel = sel;
  a.sel_ld = sel_ld;
  a.K = K;
  const int T = list ? K : (L + kPage - 1) / kPage;
  const int nc = page_attn_chunks(BH, a.G, T);
  a.chunk = (T + nc - 1) / nc;
  a.n_chunks = (T + a.chunk - 1) / a.chunk;
  a.scale_log2 = kLog2e / sqrtf((float)shape->D);
  a.out = out;
  a.lse = lse;
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + w.part_off);
  a.ml = reinterpret_cast<float*>(static_cast<char*>(ws) + w.ml_off);
  cudaStream_t st = (cudaStream_t)stream;
  const int D = shape->D;
  if (!q8) return launch_any<kBf16, true>(D, a, st);
  if (q8->format == SFI_FMT_E4M3)
    return list ? launch_any<SFI_FMT_E4M3, true>(D, a, st) : launch_any<SFI_FMT_E4M3, false>(D, a, st);
  return list ? launch_any<SFI_FMT_INT8, true>(D, a, st) : launch_any<SFI_FMT_INT8, false>(D, a, st);
}

}  // namespace

// Chunks of a (sequence, KV head) with T tiles: about four waves of two CTAs
// per SM, at least 16 tiles a chunk.
int page_attn_chunks(int BH, int G, int T) {
  const int want = std::max(1, num_sms() * 8 / BH);
  return std::max(1, std::min(want, (T + 15) / 16));
}
int page_attn_chunks_bound(int BH, int G, int Tmax) { return page_attn_chunks(BH, G, Tmax); }

}  // namespace sfi

using namespace sfi;

extern "C" {

sfi_status sfi_quant_attn(const sfi_shape* shape, const sfi_quant_kv* qkv, int32_t L, const int32_t* lens,
                          const sfi_bf16* q, float* out, float* lse, void* ws, size_t ws_bytes,
                          sfi_stream stream) {
  if (!qkv) return SFI_ERR_INVALID_ARG;
  return run(shape, nullptr, qkv, L, lens, q, nullptr, 0, 0, false, out, lse, ws, ws_bytes, stream);
}

sfi_status sfi_block_attn(const sfi_shape* shape, const sfi_paged_kv* kv, int32_t L, const int32_t* lens,
                          const sfi_bf16* q, const int32_t* sel, int32_t sel_ld, int32_t K, float* out,
                          float* lse, void* ws, size_t ws_bytes, sfi_stream stream) {
  return run(shape, kv, nullptr, L, lens, q, sel, sel_ld, K, true, out, lse, ws, ws_bytes, stream);
}

sfi_status sfi_quant_block_attn(const sfi_shape* shape, const sfi_quant_kv* qkv, int32_t L, const int32_t* lens,
                                const sfi_bf16* q, const int32_t* sel, int32_t sel_ld, int32_t K, float* out,
                                float* lse, void* ws, size_t ws_bytes, sfi_stream stream) {
  if (!qkv) return SFI_ERR_INVALID_ARG;
  return run(shape, nullptr, qkv, L, lens, q, sel, sel_ld, K, true, out, lse, ws, ws_bytes, stream);
}

}  // extern "C"
