// Decode attention over pages: all pages of an 8-bit cache, or listed pages of
// an 8-bit or a bf16 cache.
//
//   z_j = q . k_j / sqrt(D),  out = sum_j softmax(z)_j v_j
//
// Work.  A tile is one page: 16 rows of K and of V.  The tiles of all rows - a
// row being one (sequence, KV head), its tiles its pages or list entries - form
// one sequence, and every CTA takes an equal run of it, whatever the lengths
// (a row counts for some tiles more than it has, see Cfg::kRowCost); the grid is
// what the GPU holds at once.  Rows of one length that divide well get the same
// number of CTAs each instead, see launch().  A run cuts at most two rows: a row
// inside one run is finished there; the pieces of the others are merged by the
// CTA that writes the last of them, in an order that is the same whoever that is,
// or, where that would be much work for one CTA, by a second kernel.
// Within a row, warp w of the CTA takes tiles w, w + W, ...; each warp runs its
// own online softmax and the CTA merges its warps in shared memory.
//
// Bound by reading the cache at G <= 8 (at G = 16 by the latency of 414
// instructions a tile with 12 warps an SM), so the layout serves the loads: two
// sequences of 128K e4m3, 32/8 heads, 537 MB, take 89 us, 6.0 TB/s, in a short
// graph and 97 in calls that go on for half a second (at the power cap); 16 of 64K
// with 64/4 heads, 1.07 GB, 237 and 261 us.  Each thread loads exactly the bytes
// its own matrix fragments need, 32 or 16 at a time, straight into registers: the
// next tile's K while the softmax and V^T P^T of this one run, its V while the
// next S^T does.  No shared memory, no barrier and no wait that another warp has
// to end.  That works because the order of a contraction is free:
//   S^T[16 tok x 8 heads] = K[16 x D] . Q^T[D x 8]: thread (g, t) of the
//     fragment layout (g = lane / 4, t = lane % 4) holds rows g, g + 8 and any
//     D / 4 of the columns, as long as Q is laid out alike: a run of them, so
//     that a warp's load covers whole rows;
//   O^T[D x 8 heads] += V^T[D x 16] . P^T[16 x 8]: it holds tokens 2t, 2t + 1,
//     2t + 8, 2t + 9 and a run of D / 8 columns of each; two tokens' bytes are
//     interleaved into the 16-bit pairs that the fragment wants.
// (A ring of stages in shared memory, filled by asynchronous copies, took 127 us
// for the 128K e4m3 case where this took 117: its copies and reads back kept the
// shared-memory pipe busy and the warps waiting for it.)
// 8-bit codes become fp16 in registers, exactly (int8 and e4m3 both fit), and Q
// fp16 times a power of two per head; the key scale multiplies the logits, the
// value scale the tile's product.  P is split into hi + lo, which keeps 22 bits
// of it in fp16 (8-bit pages) and 16 in bf16 (bf16 rows, whose range fp16 lacks).
// The softmax reference moves only when a logit exceeds it by a margin, so most
// tiles need no rescaling and no reduction.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace sfi {
namespace {

constexpr int kBf16 = 2;            // FMT: SFI_FMT_E4M3, SFI_FMT_INT8 or this
// A warp's reference m is set `bias` below its largest logit so far (log2 units)
// and moves when a logit exceeds it by bias + kSlack.  8-bit pages, kBias: P
// reaches 2^14, inside fp16, and the largest one is at least 2^8.  What fp16 holds
// is P times pv = scale / vref (tile_math), in two parts, the second in steps of at
// least 2^-24: a weight is off by at most 2^-25 / pv, 2^-33 / pv of the largest, so
// 2^-33 on pages of the largest scale and 2^-27 at pv = 2^-6, where the factor is
// taken out.  The error times the page's values, whose size goes with pv, stays
// below 2^-33 of the largest page's.  bf16 pages: O = sum P v is as large as l times the largest |v|, which
// may be the type's largest, so the reference lies above the logits, by enough
// that l <= 1/2 over all tokens of a row (bf16 holds any P alike).
constexpr float kBias = 8.f, kSlack = 6.f;
constexpr float kNoMax = -3.4028234663852886e38f;   // m before the first logit

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
  int total;                        // units of all rows (row_units), or -1: by lens
  int quota;                        // units of a CTA's run (total >= 0)
  int row_cost;                     // units of a row besides its tiles
  int ctas;                         // of the grid
  int merge_later;                  // pieces are merged by the next kernel
  int pieces;                       // > 0: CTAs of each row, whose runs begin with the row; 0: even runs
  float scale_log2;                 // log2(e) / sqrt(D)
  float bias;                       // of the reference m below the largest logit (kBias: 8-bit pages)
  float tail_unit;                  // unit of the tail's share of O: P |v| / tail_unit stays finite (8-bit pages)
  float* out;
  float* lse;
  float* part;                      // [cta][2][G][D] mean of values: piece of the row that began before, that goes on behind
  float* ml;                        // [cta][2][G][2]
  int* arrived;                     // [B * Hkv] pieces of a row written so far; zero between calls
  int* err;
};

// HM, how the group's heads fill the 8 columns of a product: kHalf (G <= 4) has
// heads 0 .. 3 twice, the second time with the low part of P, so one product
// serves both parts; kOne (G <= 8) and kTwo (G <= 16) take hi and lo in turn.
// (G = 4 through kOne against kHalf, us: 128K int8 96.3, 93.2; D = 64 128K e4m3
// 117, 115; 128K e4m3 89.8, 90.1.)
constexpr int kMaxCtas = 3;   // CTAs per SM
enum HeadMap : int { kHalf = 0, kOne = 1, kTwo = 2 };

template <int D, int FMT, int HM>
struct Cfg {
  static constexpr int NT = HM == kTwo ? 2 : 1;         // column tiles
  static constexpr int kEl = FMT == kBf16 ? 2 : 1;
  static constexpr int kRow = D * kEl;                  // bytes of a row
  static constexpr int KJ = kRow / 64;                  // 16-byte pieces of a K row per thread
  static constexpr int KL = kRow >= 128 ? 32 : 16;      // bytes of a load of them
  static constexpr int kVB = kRow / 8;                  // bytes of a V row per thread: 8, 16 or 32
  static constexpr int VC = kVB >= 16 ? kVB / 16 : 1;   // pieces of them
  static constexpr int kTile = 16 * kRow;               // bytes of a tile of K, and of V
  // First of the four columns that thread t of a quad contributes to step k of
  // S^T, and of the two that thread g contributes to m tile k of O^T.
  static __device__ __forceinline__ int k_col(int t, int k) {
    return kEl == 2 ? (k / 4) * 64 + t * 16 + (k % 4) * 4 : KJ == 2 ? t * 32 + k * 4 : t * 16 + k * 4;
  }
  static __device__ __forceinline__ int v_col(int g, int k) { return g * (D / 8) + 2 * k; }
  // Warps and CTAs per SM: as many warps as the registers allow.  us at 128K
  // e4m3: 8 x 2 93, 7 x 2 103; blocks 128K (bf16, whose tile takes twice the
  // registers): 6 x 2 62, 5 x 2 63, 7 x 2 65; 64K x 16 heads: 4 x 3 264, 5 x 2
  // 261, 6 x 2 264, 4 x 2 294.
  static constexpr int W = NT == 2 ? 4 : FMT == kBf16 ? 6 : 8;
  static constexpr int kCtas = NT == 2 ? 3 : 2;
  static_assert(kCtas <= kMaxCtas, "the workspace has two partials for each CTA of a wave");
  // Tiles fetched into L2 ahead of their loads: one for 8-bit pages (a warp's
  // registers hold one 4 KB tile in flight, less than the latency asks for),
  // none for bf16 pages, whose tile is twice as large.  us with 0, 1, 2 ahead:
  // 128K e4m3 97, 93, 96; blocks 128K 62, 64.
  static constexpr int kAhead = FMT == kBf16 ? 0 : 1;
  // What a row costs a CTA besides its tiles, in tiles: queries and pages looked
  // up, the pipeline filled and drained, the warps merged, about 3 us (twice as
  // long a tile for G > 8).  Runs of equal tile counts alone gave the CTAs with
  // many short rows most to do: 64 sequences of 25 to 1600 tokens and 8 heads
  // took 57 us, in the order of their lengths 106; with 24 units a row, 34 and
  // 34 (12: 37, 38; 16: 36, 35).
  static constexpr int kRowCost = NT == 2 ? 12 : 24;
  // and what a second row costs a run that goes on into it
  static constexpr int kSecondRow = NT == 2 ? 8 : 16;
  static constexpr int kMerge = W * NT * 8 * (D + 8) * 4 + W * NT * 8 * 2 * 4;   // merge of the warps
  // Q fragments: registers, or (G > 8, whose accumulators take twice the
  // registers) 16 bytes of shared memory per thread, column tile and two steps.
  static constexpr bool kQShared = HM == kTwo;
  static constexpr int kQ = kQShared ? W * NT * (D / 32) * 512 : 0;
  static constexpr int kSmem = kMerge + kQ;
};

// Tiles of a row of sequence b.
template <bool LIST>
__device__ __forceinline__ int row_tiles(const PageAttnArgs& a, int b, int* err) {
  return LIST ? a.K : (seq_len(a.lens, a.L, b, err) + kPage - 1) / kPage;
}

// Units of a row: its tiles, after row_cost units for what a row costs a CTA
// besides them (see Cfg::kRowCost).
__host__ __device__ __forceinline__ int row_units(int tiles, int row_cost) { return tiles > 0 ? tiles + row_cost : 0; }

// The run of each CTA, in units, of `total` units.  A run of fewer than
// kMinQuota tiles would not fill the warps of a CTA.
constexpr int kMinQuota = 16;   // us at 1K with 8, 16, 32: attention 7.0, 7.5, 12; block decode 13, 10.9, 10.8
__host__ __device__ __forceinline__ int quota(int total, int ctas, int row_cost) {
  const int q = (int)(((unsigned)total + (unsigned)ctas - 1u) / (unsigned)ctas);
  return q > kMinQuota + row_cost ? q : kMinQuota + row_cost;
}

// Units of all rows (one warp; all lanes get it).
__device__ __forceinline__ int count_units(const PageAttnArgs& a, int lane, int* err) {
  if (a.total >= 0) return a.total;   // rows of one length
  int t = 0;
  for (int i = lane; i < a.B; i += 32) t += row_units(row_tiles<false>(a, i, err), a.row_cost);
  return (int)__reduce_add_sync(0xffffffffu, (unsigned)t) * a.Hkv;
}

// The sequence whose rows hold unit `pos` (< total) and the first unit of its
// rows (one warp; all lanes get both).
template <bool LIST>
__device__ __forceinline__ void find_sequence(const PageAttnArgs& a, int pos, int lane, int& b, int& first) {
  if (a.total >= 0) {
    const unsigned per = (unsigned)a.total / (unsigned)a.B;
    b = (int)((unsigned)pos / per);
    first = (int)per * b;
    return;
  }
  int base = 0;
  for (int i0 = 0; i0 < a.B; i0 += 32) {
    const int i = i0 + lane;
    const int v = i < a.B ? row_units(row_tiles<LIST>(a, i, nullptr), a.row_cost) * a.Hkv : 0;
    int x = v;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, sh);
      if (lane >= sh) x += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + x > pos);
    if (hit) {
      const int l = __ffs(hit) - 1;
      b = i0 + l;
      first = base + __shfl_sync(0xffffffffu, x - v, l);
      return;
    }
    base += __shfl_sync(0xffffffffu, x, 31);
  }
  b = a.B;   // not reached for pos < total
  first = base;
}

struct Tile {
  int page;         // >= 0; -1: nothing; -2: the tail
  int rows;         // valid rows
  float ks, vs;
};

// 16 or 8 bytes of the cache, read once: kept in program order, so that a load
// stays where the code issues it, ahead of the work it overlaps.
__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ void ld32(const uint8_t* p, uint4& x, uint4& y) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w), "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
               : "l"(p));
}
__device__ __forceinline__ uint4 ld8(const uint8_t* p) {
  uint4 r = make_uint4(0, 0, 0, 0);
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// D += A * B, m16n8k16, fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D += A * B, or D = A * B.
template <bool F16, bool ADD>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (ADD) {
    if constexpr (F16) mma_f16_16816(d, a, b0, b1);
    else mma_bf16_16816(d, a, b0, b1);
  } else if constexpr (F16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  }
}

// Codes in bytes 0, 1 of v -> lo and bytes 2, 3 -> hi, as fp16 pairs, exactly.
// e4m3: the hardware conversion.  int8: x + 128 in the low byte of 0x6400 is
// 1024 + 128 + x in fp16, less 1152.
template <int FMT>
__device__ __forceinline__ void to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == SFI_FMT_INT8) {
    const uint32_t u = v ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 k = __float2half2_rn(1152.f);
    const __half2 e = __hsub2(*reinterpret_cast<const __half2*>(&a), k);
    const __half2 f = __hsub2(*reinterpret_cast<const __half2*>(&b), k);
    lo = *reinterpret_cast<const uint32_t*>(&e);
    hi = *reinterpret_cast<const uint32_t*>(&f);
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
  }
}

__device__ __forceinline__ uint32_t word(const uint4& x, int w) { return w == 0 ? x.x : w == 1 ? x.y : w == 2 ? x.z : x.w; }

// The state of one warp: reference m (log2 units) and this thread's share of
// the sum for heads 2t, 2t + 1 of each head tile, and O^T in units of vref.
template <int D, int NT>
struct State {
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];
  float vref, vinv;   // and 1 / vref
};

template <int D, int NT>
__device__ __forceinline__ void scale_o(State<D, NT>& st, float f) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[nt][k][i] *= f;
}

// One tile from its fragments: kf(step, a) and vf(step, a) fill the A operands
// of S^T and O^T, qf(column tile, step, b0, b1) the B operand of S^T; between()
// runs once K is used up.  zf: log2 units per unit of S^T, per head; vs: the
// value scale, or the tail's unit; bias: of the reference; rows: valid rows.  F16: fp16 operands (8-bit pages), else bf16.
// SCALED: the cache has value scales.  UNROLL: of the rescaling of O, 1 or 2; rolled
// it costs the list kernel of 16 heads fewer registers (64K, 820 blocks, 64/4 heads:
// 93.5 -> 90.1 us), the one without a list runs better unrolled (64K 251.9, 245.4).
template <int D, int HM, bool F16, bool SCALED, int UNROLL, class KF, class QF, class BW, class VF, int NT>
__device__ __forceinline__ void tile_math(State<D, NT>& st, const float (&zf)[NT][2], float vs, float bias, int rows,
                                          int lane, KF kf, QF qf, BW between, VF vf) {
  float s[NT][4], x[NT][4];
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    uint32_t a[4];
    kf(k, a);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t b0, b1;
      qf(nt, k, b0, b1);
      if (k == 0) mma16<F16, false>(s[nt], a, b0, b1);
      else if (k == 1) mma16<F16, false>(x[nt], a, b0, b1);
      else if (k % 2 == 0) mma16<F16, true>(s[nt], a, b0, b1);
      else mma16<F16, true>(x[nt], a, b0, b1);
    }
  }
  between();
  bool grow = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[nt][i] += x[nt][i];
      x[nt][i] = fmaf(s[nt][i], zf[nt][i & 1], -st.m[nt][i & 1]);   // one rounding, of the difference
      if (!F16 && rows < kPage && (lane >> 2) + 8 * (i >> 1) >= rows) x[nt][i] = -INFINITY;   // 8-bit pages are full
      grow |= x[nt][i] > bias + kSlack;
    }
  if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float z = -INFINITY;
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (x[nt][j + 2 * r] != -INFINITY) z = fmaxf(z, s[nt][j + 2 * r] * zf[nt][j]);
#pragma unroll
        for (int sh = 4; sh <= 16; sh <<= 1) z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, sh));
        const float mn = fmaxf(st.m[nt][j], z - bias);
        const float al = fast_exp2(st.m[nt][j] - mn);
        st.m[nt][j] = mn;
        st.l[nt][j] *= al;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          st.o[nt][k][j] *= al;
          st.o[nt][k][j + 2] *= al;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (x[nt][j + 2 * r] != -INFINITY) x[nt][j + 2 * r] = fmaf(s[nt][j + 2 * r], zf[nt][j], -mn);
      }
  }
  // The value scale multiplies P, relative to vref so that fp16 holds it: vref
  // follows the largest scale seen (within a factor of 2); a page whose scale
  // is 2^6 and more below it, which fp16 would hold to fewer than 2^-27, has its
  // product scaled instead.
  float pv = 1.f;
  bool apart = false;
  if constexpr (SCALED) {
    if (!(vs <= 2.f * st.vref)) {   // NaN too
      // O times vref / vs: in two steps, since the quotient alone may leave fp32's
      // range, the first being the one that keeps the product inside it
      st.vinv = __fdiv_rn(1.f, vs);
      const bool large = vs >= 1.f;
#pragma unroll UNROLL
      for (int i = 0; i < 2; ++i) scale_o(st, (i == 0) == large ? st.vinv : st.vref);
      st.vref = vs;
    }
    pv = F16 ? vs * st.vinv : st.vinv;   // the tail's values have no scale
    // the same in every lane; the vote lets the compiler branch
    if (F16) apart = __any_sync(0xffffffffu, pv < 0.015625f);
  }
  uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float p0 = fast_exp2(x[nt][2 * r]), p1 = fast_exp2(x[nt][2 * r + 1]);
      st.l[nt][0] += p0;
      st.l[nt][1] += p1;
      if constexpr (SCALED) {
        const float f = apart ? 1.f : pv;
        p0 *= f;
        p1 *= f;
      }
      const uint32_t h = F16 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
      const float2 f = F16 ? unpack_f16x2(h) : unpack_bf16x2(h);
      const uint32_t q = F16 ? pack_f16x2(p0 - f.x, p1 - f.y) : pack_bf16x2(p0 - f.x, p1 - f.y);
      if constexpr (HM == kHalf) {
        hi[nt][r] = movmatrix_trans((lane & 2) ? q : h);
      } else {
        hi[nt][r] = movmatrix_trans(h);
        lo[nt][r] = movmatrix_trans(q);
      }
    }
  if (SCALED && F16 && apart) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t a[4];
      vf(k, a);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float c[4];
        mma16<F16, false>(c, a, hi[nt][0], hi[nt][1]);
        if constexpr (HM != kHalf) mma16<F16, true>(c, a, lo[nt][0], lo[nt][1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) st.o[nt][k][i] = fmaf(c[i] * vs, st.vinv, st.o[nt][k][i]);   // pv may be subnormal
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t a[4];
      vf(k, a);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma16<F16, true>(st.o[nt][k], a, hi[nt][0], hi[nt][1]);
        if constexpr (HM != kHalf) mma16<F16, true>(st.o[nt][k], a, lo[nt][0], lo[nt][1]);
      }
    }
  }
}

__device__ __forceinline__ void add_scaled(float4& o, float f, const float4& x) {
  o.x = fmaf(f, x.x, o.x);
  o.y = fmaf(f, x.y, o.y);
  o.z = fmaf(f, x.z, o.z);
  o.w = fmaf(f, x.w, o.w);
}

// 1 / sum of the weights of a merge, off by at most 2^-23 of itself (sums lie
// between 2^-50 and 2^50; a division in fp32's full range took 0.5 us of a short
// call); nothing to attend to: 0.
__device__ __forceinline__ float inverse(float l) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(l));
  return l == 0.f ? 0.f : r;
}

// Columns d .. d + 3 of an output row, the mean o of the values, and its
// log-sum-exp from (m, l); l = 0: nothing to attend to.  l's exponent joins m
// first, so that the logarithm's error is not one of a large l's.
template <int D>
__device__ __forceinline__ void write_out(const PageAttnArgs& a, size_t row, int d, float M, float l, const float4& o) {
  const bool none = l == 0.f;
  *reinterpret_cast<float4*>(a.out + row * D + d) = none ? make_float4(0.f, 0.f, 0.f, 0.f) : o;
  if (d == 0 && a.lse) {
    const uint32_t u = __float_as_uint(l);
    const float e = (float)((int)(u >> 23) - 127);
    const float lse = ((M + e) + fast_log2(__uint_as_float((u & 0x7fffffu) | 0x3f800000u))) * kLn2;
    a.lse[row] = none ? -INFINITY : l != l ? l : lse;
  }
}

constexpr int kMaxGroups = 8;

// The CTAs with a piece of a row: its first unit is row0, its tiles T > 0.
__device__ __forceinline__ void row_ctas(const PageAttnArgs& a, int b, int h, int T, int row0, int run, int& c0, int& c1) {
  if (a.pieces > 0) {
    c0 = (b * a.Hkv + h) * a.pieces;
    c1 = c0 + a.pieces - 1;
  } else {
    c0 = (int)((unsigned)(row0 + a.row_cost) / (unsigned)run);
    c1 = (int)((unsigned)(row0 + T + a.row_cost - 1) / (unsigned)run);
  }
}

// Tiles [t0, t1) of the T tiles of row (b, h), by the whole CTA: the row's
// output, or (not the whole row) its piece, and the output too if that is the
// last.  c0, c1: the first and last CTA with a piece of the row.
template <int D, int FMT, int HM, bool LIST>
__device__ __forceinline__ void attend_row(const PageAttnArgs& a, uint8_t* smem, int b, int h, int len, int T, int t0,
                                           int t1, int c0, int c1) {
  using C = Cfg<D, FMT, HM>;
  constexpr int NT = C::NT, W = C::W, KJ = C::KJ, VC = C::VC;
  constexpr int kUnroll = LIST && HM == kTwo ? 1 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int bh = b * a.Hkv + h;
  const int blocks = (len + kPage - 1) / kPage;

  // queries of the group: B operands of S^T, in the column order of the K
  // fragments (zero for heads past G).  8-bit pages: fp16, each head times the
  // power of two that takes its largest value into [2^14, 2^15) (an element
  // below 2^-39 of that loses bits); zq undoes it.
  uint32_t qb[NT][D / 16][2];
  uint4* qs = reinterpret_cast<uint4*>(smem + C::kMerge) + warp * NT * (D / 32) * 32 + lane;
  float zq[NT][2];
  auto q_at = [&](int nt, int k) {   // four columns of the head of column nt * 8 + g
    const int n = HM == kHalf ? g & 3 : nt * 8 + g;
    if (n >= a.G) return make_uint2(0, 0);
    return __ldg(reinterpret_cast<const uint2*>(a.q + ((size_t)b * a.Hq + h * a.G + n) * D + C::k_col(t, k)));
  };
  // ahead of the look-up; converted behind the first loads of K and V
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint2 x = q_at(nt, k);
      qb[nt][k][0] = x.x;
      qb[nt][k][1] = x.y;
    }

  // Tiles of this warp: t0 + warp + W * i, i < n.  Lane l looks up tile i0 + l of
  // a batch of 32: block, page and scales.
  const int n = t1 - t0 > warp ? (t1 - t0 - warp + W - 1) / W : 0;
  Tile mine{-1, 0, 0.f, 0.f};
  auto look_up = [&](int i0) {
    mine = Tile{-1, 0, 0.f, 0.f};
    const int i = i0 + lane;
    const int tile = t0 + warp + W * i;
    const int blk = i >= n ? -1 : LIST ? __ldg(a.sel + (size_t)bh * a.sel_ld + tile) : tile;
    if ((unsigned)blk < (unsigned)blocks) {
      mine.rows = min(kPage, len - blk * kPage);
      if (FMT != kBf16 && mine.rows < kPage) {
        mine.page = -2;
      } else {
        const int page = __ldg(a.pt + (size_t)b * a.max_pages + blk);
        if ((unsigned)page < (unsigned)a.num_pages) {
          mine.page = page;
          if (FMT != kBf16) {
            mine.ks = __ldg(a.ks + (size_t)page * a.Hkv + h);
            mine.vs = __ldg(a.vs + (size_t)page * a.Hkv + h);
          }
        } else {
          latch_error(a.err, SFI_ERR_DEVICE_CHECK, kSitePageAttn);
          mine.rows = 0;
        }
      }
    }
    // the tail's rows are not loaded ahead of their use: bring them close
    if (FMT != kBf16 && __any_sync(0xffffffffu, mine.page == -2)) {
      const char* kt = reinterpret_cast<const char*>(a.k_tail + (size_t)bh * (kPage * D));
      const char* vt = reinterpret_cast<const char*>(a.v_tail + (size_t)bh * (kPage * D));
      for (int o = lane * 128; o < kPage * D * 2; o += 32 * 128) {
        asm volatile("prefetch.global.L2 [%0];" ::"l"(kt + o));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(vt + o));
      }
    }
  };
  // The warp brings a tile into L2 kAhead tiles before it loads it.
  auto fetch = [&](int j) {
    const int page = __shfl_sync(0xffffffffu, mine.page, j);
    if (page < 0) return;
    const size_t off = ((size_t)page * a.Hkv + h) * C::kTile;
#pragma unroll
    for (int o = (lane & 15) * 128; o < C::kTile; o += 2048)
      asm volatile("prefetch.global.L2 [%0];" ::"l"((lane < 16 ? a.k : a.v) + off + o));
  };
  auto tile_at = [&](int i) {
    Tile x{-1, 0, 0.f, 0.f};
    if (i >= n) return x;
    if ((i & 31) == 0) {
      look_up(i);
      for (int j = 1; j <= C::kAhead; ++j) fetch(j);
    } else if (C::kAhead > 0 && (i & 31) + C::kAhead < 32) {
      fetch((i & 31) + C::kAhead);
    }
    x.page = __shfl_sync(0xffffffffu, mine.page, i & 31);
    x.rows = __shfl_sync(0xffffffffu, mine.rows, i & 31);
    return x;
  };
  // the scales of tile i, before tile_at(i + 1): their loads are not waited for
  // ahead of the first loads of K and V
  auto scales_at = [&](Tile& x, int i) {
    if (FMT != kBf16) {
      x.ks = __shfl_sync(0xffffffffu, mine.ks, i & 31);
      x.vs = __shfl_sync(0xffffffffu, mine.vs, i & 31);
    }
  };
  uint4 kx[2 * KJ], vx[4 * VC];
  const uint8_t* k0 = a.k + (size_t)h * C::kTile + g * C::kRow + t * C::KL;
  const uint8_t* v0 = a.v + (size_t)h * C::kTile + 2 * t * C::kRow + g * C::kVB;
  auto load_k = [&](const Tile& x) {
    const uint8_t* p = k0 + (size_t)x.page * a.Hkv * C::kTile;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint8_t* at = p + r * 8 * C::kRow;
      if (FMT == kBf16 && g + 8 * r >= x.rows) {
#pragma unroll
        for (int j = 0; j < KJ; ++j) kx[r * KJ + j] = make_uint4(0, 0, 0, 0);
      } else if constexpr (C::KL == 32) {
#pragma unroll
        for (int j = 0; j < KJ; j += 2) ld32(at + j * 64, kx[r * KJ + j], kx[r * KJ + j + 1]);
      } else {
        kx[r] = ld16(at);
      }
    }
  };
  auto load_v = [&](const Tile& x) {
    const uint8_t* p = v0 + (size_t)x.page * a.Hkv * C::kTile;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = (i & 1) + 8 * (i >> 1);
      const uint8_t* at = p + tok * C::kRow;
      if (FMT == kBf16 && 2 * t + tok >= x.rows) {
#pragma unroll
        for (int c = 0; c < VC; ++c) vx[i * VC + c] = make_uint4(0, 0, 0, 0);
      } else if constexpr (C::kVB == 32) {
        ld32(at, vx[2 * i], vx[2 * i + 1]);
      } else if constexpr (C::kVB == 16) {
        vx[i] = ld16(at);
      } else {
        vx[i] = ld8(at);
      }
    }
  };

  State<D, NT> st;
  st.vref = FMT == kBf16 ? 1.f : 1.17549435e-38f;   // the smallest normal: any scale takes its place
  st.vinv = FMT == kBf16 ? 1.f : 8.50705917e37f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      st.m[nt][j] = kNoMax;
      st.l[nt][j] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[nt][k][i] = 0.f;
  }

  auto q_regs = [&](int nt, int k, uint32_t& b0, uint32_t& b1) {
    if constexpr (C::kQShared) {
      const uint4 x = qs[(nt * (D / 32) + k / 2) * 32];   // this thread's own words
      b0 = k % 2 ? x.z : x.x;
      b1 = k % 2 ? x.w : x.y;
    } else {
      b0 = qb[nt][k][0];
      b1 = qb[nt][k][1];
    }
  };
  Tile cur = tile_at(0);
  if (cur.page >= 0) {
    load_k(cur);
    load_v(cur);
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t(&q)[D / 16][2] = qb[nt];
    zq[nt][0] = zq[nt][1] = a.scale_log2;
    if constexpr (FMT != kBf16) {
      uint32_t am = 0;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) am = __vmaxu2(am, __vmaxu2(q[k][0] & 0x7fff7fffu, q[k][1] & 0x7fff7fffu));
      am = max(am & 0xffffu, am >> 16);
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      // biased exponent of the head's largest value; up = 2^(14 - exponent)
      const int e = (int)(am >> 7);
      const int up = e == 0xff || am == 0 ? 127 : min(127 + 14 - (e - 127), 253);
      const float f = __uint_as_float((uint32_t)up << 23), inv = __uint_as_float((uint32_t)(254 - up) << 23);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 x = unpack_bf16x2(q[k][i]);
          q[k][i] = pack_f16x2(x.x * f, x.y * f);
        }
#pragma unroll
      for (int j = 0; j < 2; ++j) zq[nt][j] *= __shfl_sync(0xffffffffu, inv, (2 * t + j) * 4);
    }
    if constexpr (C::kQShared) {
#pragma unroll
      for (int k = 0; k < D / 16; k += 2)
        qs[(nt * (D / 32) + k / 2) * 32] = make_uint4(q[k][0], q[k][1], q[k + 1][0], q[k + 1][1]);
    }
  }
  for (int i = 0; i < n; ++i) {
    scales_at(cur, i);
    const Tile nxt = tile_at(i + 1);
    auto next_k = [&]() {
      if (nxt.page >= 0) load_k(nxt);
    };
    if (cur.page >= 0) {
      if constexpr (FMT == kBf16) {
        tile_math<D, HM, false, false, 2>(
            st, zq, 1.f, a.bias, cur.rows, lane,
            [&](int k, uint32_t (&f)[4]) {
              const int w = (k % 2) * 2;
              f[0] = word(kx[k / 2], w);
              f[1] = word(kx[KJ + k / 2], w);
              f[2] = word(kx[k / 2], w + 1);
              f[3] = word(kx[KJ + k / 2], w + 1);
            },
            q_regs, next_k,
            [&](int k, uint32_t (&f)[4]) {
              const int c = k / 4, w = k % 4;
              const uint32_t x0 = word(vx[c], w), x1 = word(vx[VC + c], w);
              const uint32_t x2 = word(vx[2 * VC + c], w), x3 = word(vx[3 * VC + c], w);
              f[0] = __byte_perm(x0, x1, 0x5410);
              f[1] = __byte_perm(x0, x1, 0x7632);
              f[2] = __byte_perm(x2, x3, 0x5410);
              f[3] = __byte_perm(x2, x3, 0x7632);
            });
      } else {
        float zf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) zf[nt][j] = zq[nt][j] * cur.ks;
        tile_math<D, HM, true, true, kUnroll>(
            st, zf, cur.vs, kBias, kPage, lane,
            [&](int k, uint32_t (&f)[4]) {
              to_f16<FMT>(word(kx[k / 4], k % 4), f[0], f[2]);
              to_f16<FMT>(word(kx[KJ + k / 4], k % 4), f[1], f[3]);
            },
            q_regs, next_k,
            [&](int k, uint32_t (&f)[4]) {
              // the two tokens' bytes of column d, then of column d + 1
              const uint32_t sel = k % 2 ? 0x7362 : 0x5140;
              const int w = k / 2;
              to_f16<FMT>(__byte_perm(word(vx[0], w), word(vx[1], w), sel), f[0], f[1]);
              to_f16<FMT>(__byte_perm(word(vx[2], w), word(vx[3], w), sel), f[2], f[3]);
            });
      }
    } else {
      next_k();
    }
    if (FMT != kBf16 && cur.page == -2) {
      // the bf16 rows of the page that is not full, straight from memory, in
      // the column orders of the 8-bit fragments
      const __nv_bfloat16* kt = a.k_tail + (size_t)bh * (kPage * D);
      const __nv_bfloat16* vt = a.v_tail + (size_t)bh * (kPage * D);
      const int tail_rows = cur.rows;
      float zt[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) zt[nt][0] = zt[nt][1] = a.scale_log2;
      tile_math<D, HM, false, true, kUnroll>(
          st, zt, a.tail_unit, kBias, tail_rows, lane,
          [&](int k, uint32_t (&f)[4]) {
            const int d = C::k_col(t, k);
            uint2 x = make_uint2(0, 0), y = make_uint2(0, 0);
            if (g < tail_rows) x = __ldg(reinterpret_cast<const uint2*>(kt + g * D + d));
            if (g + 8 < tail_rows) y = __ldg(reinterpret_cast<const uint2*>(kt + (g + 8) * D + d));
            f[0] = x.x;
            f[1] = y.x;
            f[2] = x.y;
            f[3] = y.y;
          },
          [&](int nt, int k, uint32_t& b0, uint32_t& b1) {
            const uint2 x = q_at(nt, k);
            b0 = x.x;
            b1 = x.y;
          },
          []() {},
          [&](int k, uint32_t (&f)[4]) {
            const int d = C::v_col(g, k);
            uint32_t x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int tok = 2 * t + (r & 1) + 8 * (r >> 1);
              x[r] = tok < tail_rows ? __ldg(reinterpret_cast<const uint32_t*>(vt + tok * D + d)) : 0u;
            }
            f[0] = __byte_perm(x[0], x[1], 0x5410);
            f[1] = __byte_perm(x[0], x[1], 0x7632);
            f[2] = __byte_perm(x[2], x[3], 0x5410);
            f[3] = __byte_perm(x[2], x[3], 0x7632);
          });
    }
    if (nxt.page >= 0) load_v(nxt);
    cur = nxt;
  }

  // Merge of the CTA's warps: O / l of each head, row of D floats padded by 8,
  // then (m, l) of each head.  From here on everything is a mean of values with
  // weights that add up to 1: it stays finite when the values are the type's
  // largest, where O and l apart would not.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int sh = 4; sh <= 16; sh <<= 1) st.l[nt][j] += __shfl_xor_sync(0xffffffffu, st.l[nt][j], sh);
  constexpr int kLd = D + 8;
  float* so = reinterpret_cast<float*>(smem);
  float* sml = so + W * NT * 8 * kLd;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float r = inverse(st.l[nt][j]);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        *reinterpret_cast<float2*>(so + (size_t)(warp * NT * 8 + nt * 8 + 2 * t + j) * kLd + C::v_col(g, k)) =
            make_float2(st.o[nt][k][j] * r * st.vref, st.o[nt][k][j + 2] * r * st.vref);
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
  const bool whole = t0 == 0 && t1 == T;
  const int item = blockIdx.x * 2 + (t0 > 0 ? 0 : 1);
  for (int e = threadIdx.x; e < a.G * (D / 4); e += W * 32) {
    const int n_ = e / (D / 4), d = e % (D / 4) * 4;
    float M = kNoMax;
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, sml[(w * NT * 8 + n_) * 2]);
    float l = 0.f, weight[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 ml = *reinterpret_cast<const float2*>(sml + (w * NT * 8 + n_) * 2);
      weight[w] = fast_exp2(ml.x - M) * ml.y;
      l += weight[w];
    }
    const float r = inverse(l);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = weight[w] * r;
      add_scaled(o, f, *reinterpret_cast<const float4*>(so + (w * NT * 8 + n_) * kLd + d));
      if (HM == kHalf) add_scaled(o, f, *reinterpret_cast<const float4*>(so + (w * 8 + n_ + 4) * kLd + d));
    }
    if (whole) {
      write_out<D>(a, (size_t)b * a.Hq + h * a.G + n_, d, M, l, o);
    } else {
      *reinterpret_cast<float4*>(a.part + ((size_t)item * a.G + n_) * D + d) = o;
      if (d == 0) *reinterpret_cast<float2*>(a.ml + ((size_t)item * a.G + n_) * 2) = make_float2(M, l);
    }
  }
  if (whole) return;

  if (a.merge_later) return;

  // The CTA that writes a row's last piece merges them all.
  __syncthreads();   // the piece is written
  int* last = reinterpret_cast<int*>(sml);   // the warps' (m, l) are used up
  if (threadIdx.x == 0) {
    // releases the CTA's piece (written before the barrier), acquires the others'
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(a.arrived + bh) : "memory");
    const bool all = before == (uint32_t)(c1 - c0);
    if (all) a.arrived[bh] = 0;   // for the next call
    // more than the row has pieces: the workspace was not zero
    if (before > (uint32_t)(c1 - c0)) latch_error(a.err, SFI_ERR_DEVICE_CHECK, kSiteArrived);
    *last = all;
  }
  __syncthreads();
  if (!*last) return;
  // slots of 4 columns; threads beyond them share the pieces out in groups
  const int slots = a.G * (D / 4), groups = max(1, min(W * 32 / slots, kMaxGroups));
  for (int e = threadIdx.x; e < slots * groups; e += W * 32) {
    const int grp = e / slots, slot = e % slots, n_ = slot / (D / 4), d = slot % (D / 4) * 4;
    float M = kNoMax, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // four pieces' loads at a time, the last ones' too: one wait (us at 8K e4m3
    // with the last ones in turn and this: 21.0, 20.3)
    for (int c = c0 + grp; c <= c1; c += 4 * groups) {
      float2 ml[4];
      float4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ci = c + i * groups;
        const size_t r = ((size_t)ci * 2 + (ci > c0 ? 0 : 1)) * a.G + n_;   // only the first piece begins inside its run
        ml[i] = ci <= c1 ? __ldcg(reinterpret_cast<const float2*>(a.ml + r * 2)) : make_float2(kNoMax, 0.f);
        x[i] = ci <= c1 ? __ldcg(reinterpret_cast<const float4*>(a.part + r * D + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      const float mn = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
      float f = l * fast_exp2(M - mn), sum = f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ml[i].y *= fast_exp2(ml[i].x - mn);
        sum += ml[i].y;
      }
      const float r = inverse(sum);
      f *= r;
      o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
      for (int i = 0; i < 4; ++i) add_scaled(o, ml[i].y * r, x[i]);
      l = sum;
      M = mn;
    }
    if (groups == 1) {
      write_out<D>(a, (size_t)b * a.Hq + h * a.G + n_, d, M, l, o);
    } else {   // one pass of the loop: slots * groups <= threads
      float* g_ = so + e * 8;
      *reinterpret_cast<float4*>(g_) = o;
      *reinterpret_cast<float2*>(g_ + 4) = make_float2(M, l);
    }
  }
  if (groups == 1) return;
  __syncthreads();
  for (int slot = threadIdx.x; slot < slots; slot += W * 32) {
    float M = kNoMax, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < groups; ++i) M = fmaxf(M, so[(i * slots + slot) * 8 + 4]);
    for (int i = 0; i < groups; ++i) {
      const float* g_ = so + (i * slots + slot) * 8;
      l += fast_exp2(g_[4] - M) * g_[5];
    }
    const float r = inverse(l);
    for (int i = 0; i < groups; ++i) {
      const float* g_ = so + (i * slots + slot) * 8;
      add_scaled(o, fast_exp2(g_[4] - M) * g_[5] * r, *reinterpret_cast<const float4*>(g_));
    }
    write_out<D>(a, (size_t)b * a.Hq + h * a.G + slot / (D / 4), slot % (D / 4) * 4, M, l, o);
  }
}

template <int D, int FMT, int HM, bool LIST>
__global__ void __launch_bounds__(Cfg<D, FMT, HM>::W * 32, Cfg<D, FMT, HM>::kCtas)
    page_attn_kernel(const __grid_constant__ PageAttnArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_enter();   // the next launch may come up while this one runs; it waits before it touches memory
  // this CTA's run: `left` units from unit v0 of row (b, h) on, whose first unit is row0
  int b, h, v0, left, row0 = 0, run;
  if (a.pieces > 0) {
    const int T = row_tiles<LIST>(a, 0, nullptr);
    const unsigned row = blockIdx.x / (unsigned)a.pieces;
    run = a.quota;
    b = (int)(row / (unsigned)a.Hkv);
    h = (int)row - b * a.Hkv;
    v0 = a.row_cost + (int)(blockIdx.x - row * a.pieces) * run;
    left = min(run, T + a.row_cost - v0);
  } else {
    const int total = count_units(a, lane, warp == 0 ? a.err : nullptr);
    run = a.total >= 0 ? a.quota : quota(total, a.ctas, a.row_cost);
    const int pos = (int)min((long long)run * blockIdx.x, (long long)total);
    left = min(run, total - pos);
    if (left > 0) {
      int first;
      find_sequence<LIST>(a, pos, lane, b, first);
      const int V = row_units(row_tiles<LIST>(a, b, nullptr), a.row_cost);
      h = (int)((unsigned)(pos - first) / (unsigned)V);
      row0 = first + h * V;
      v0 = pos - row0;
    }
  }
  for (; left > 0; ++b, h = 0) {   // sequences
    const int len = seq_len(a.lens, a.L, b, LIST && a.lens && warp == 0 ? a.err : nullptr);
    const int T = LIST ? a.K : (len + kPage - 1) / kPage;
    if (T == 0) continue;
    const int V = row_units(T, a.row_cost);
    for (; h < a.Hkv && left > 0; ++h) {   // rows
      const int v1 = min(V, v0 + left);
      if (v1 > a.row_cost) {   // else none of its tiles
        int c0, c1;
        row_ctas(a, b, h, T, row0, run, c0, c1);
        attend_row<D, FMT, HM, LIST>(a, smem, b, h, len, T, max(0, v0 - a.row_cost), v1 - a.row_cost, c0, c1);
        __syncthreads();   // the row's shared memory is free
      }
      left -= v1 - v0;
      row0 += V;
      v0 = 0;
    }
  }
  if (a.total < 0) {   // the outputs of empty sequences
    for (int i = blockIdx.x; i < a.B; i += gridDim.x) {
      if (row_tiles<LIST>(a, i, nullptr) > 0) continue;
      for (int e = threadIdx.x; e < a.Hq * (D / 4); e += blockDim.x)
        write_out<D>(a, (size_t)i * a.Hq + e / (D / 4), e % (D / 4) * 4, 0.f, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
    }
  }
}

// Merge of the pieces of rows, a CTA per query head.  The pieces' (m, l) come in
// first, all at once; then each thread adds up four columns over its share of the
// pieces, in an order that the sizes alone give, and no load waits for another.
constexpr int kMergeThreads = 256;
constexpr int merge_smem(int pieces) { return kMergeThreads * 16 + pieces * 8 + 64; }   // acc, ml, group_l

template <int D, bool LIST>
__global__ void __launch_bounds__(kMergeThreads) page_merge_kernel(const __grid_constant__ PageAttnArgs a) {
  grid_dep_enter();
  extern __shared__ __align__(16) float merge_sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head = blockIdx.x, b = head / a.Hq, hq = head - b * a.Hq, h = hq / a.G, n = hq - h * a.G;
  const int T = row_tiles<LIST>(a, b, nullptr);
  if (T == 0) return;   // written by the attention kernel, as are rows in one piece
  int row0 = 0, run = a.quota;
  if (a.pieces == 0) {
    const int V = row_units(T, a.row_cost);
    if (a.total >= 0) {
      row0 = (b * a.Hkv + h) * V;
    } else {
      int before = 0, all = 0;
      for (int i = lane; i < a.B; i += 32) {
        const int u = row_units(row_tiles<LIST>(a, i, nullptr), a.row_cost);
        all += u;
        if (i < b) before += u;
      }
      row0 = (int)__reduce_add_sync(0xffffffffu, (unsigned)before) * a.Hkv + h * V;
      run = quota((int)__reduce_add_sync(0xffffffffu, (unsigned)all) * a.Hkv, a.ctas, a.row_cost);
    }
  }
  int c0, c1;
  row_ctas(a, b, h, T, row0, run, c0, c1);
  if (c0 == c1) return;
  const int P = c1 - c0 + 1;
  float4* acc = reinterpret_cast<float4*>(merge_sm);               // [groups][D / 4]
  float2* ml = reinterpret_cast<float2*>(acc + kMergeThreads);     // [P] (m, l)
  __shared__ float2 warp_max[kMergeThreads / 32];
  // only the first piece begins inside its CTA's run
  auto at = [&](int c) { return ((size_t)(c0 + c) * 2 + (c > 0 ? 0 : 1)) * a.G + n; };
  float M = kNoMax, top = 0.f;   // the largest m and l
  for (int c = tid; c < P; c += kMergeThreads) {
    ml[c] = __ldcg(reinterpret_cast<const float2*>(a.ml + at(c) * 2));
    M = fmaxf(M, ml[c].x);
    top = fmaxf(top, ml[c].y);
  }
#pragma unroll
  for (int sh = 16; sh >= 1; sh >>= 1) {
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, sh));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
  }
  if (lane == 0) warp_max[warp] = make_float2(M, top);
  __syncthreads();
  for (int w = 0; w < kMergeThreads / 32; ++w) {
    M = fmaxf(M, warp_max[w].x);
    top = fmaxf(top, warp_max[w].y);
  }
  // weights times 2^-k, which keeps their sum at or below 1
  const int k = (int)(__float_as_uint(top) >> 23) - 126 + (32 - __clz(P));
  const float unit = __uint_as_float((uint32_t)(127 - k) << 23);
  constexpr int kSlots = D / 4, kGroups = kMergeThreads / kSlots;
  const int grp = tid / kSlots, slot = tid % kSlots;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;   // of this group's pieces
#pragma unroll 8
  for (int c = grp; c < P; c += kGroups) {
    const float f = fast_exp2(ml[c].x - M) * (ml[c].y * unit);
    l += f;
    add_scaled(o, f, __ldcg(reinterpret_cast<const float4*>(a.part + at(c) * D + slot * 4)));
  }
  acc[tid] = o;
  float* group_l = reinterpret_cast<float*>(ml + P);
  if (slot == 0) group_l[grp] = l;
  __syncthreads();
  if (tid >= kSlots) return;
  for (int i = 1; i < kGroups; ++i) add_scaled(o, 1.f, acc[i * kSlots + slot]);
  l = 0.f;
  for (int i = 0; i < kGroups; ++i) l += group_l[i];
  const float r = inverse(l);
  o = make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
  l *= __uint_as_float((uint32_t)(127 + k) << 23);
  write_out<D>(a, (size_t)b * a.Hq + hq, slot * 4, M, l, o);
}

// Rows of one length get the same number of CTAs each where that makes no run
// longer by more than kSecondRow.  Measured, us, even runs against
// this: 1K int8 10.6 -> 7.5, 8K e4m3 25.3 -> 21.8, 128K e4m3 94.5 -> 89.8.
template <int D, int FMT, int HM, bool LIST>
sfi_status launch(PageAttnArgs& a, cudaStream_t st) {
  using C = Cfg<D, FMT, HM>;
  auto k = page_attn_kernel<D, FMT, HM, LIST>;
  static DeviceOnce once;
  if (!once.done()) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (!once.mark(e)) return cuda_status(e);
  }
  const int T = LIST ? a.K : (a.L + kPage - 1) / kPage;
  const long long total = (long long)a.B * a.Hkv * row_units(T, C::kRowCost);
  if (total > 0x7fffffffLL) return SFI_ERR_SHAPE;
  // one wave, fewer CTAs where the tiles would not give each kMinQuota
  const int wave = num_sms() * C::kCtas;
  int ctas = (int)std::min((long long)wave, (total + kMinQuota + C::kRowCost - 1) / (kMinQuota + C::kRowCost));
  a.total = !LIST && a.lens ? -1 : (int)total;
  a.quota = quota((int)total, ctas, C::kRowCost);
  a.row_cost = C::kRowCost;
  a.pieces = 0;
  const int rows = a.B * a.Hkv;
  if (a.total >= 0 && rows <= wave) {
    const int p = wave / rows;
    const int run = std::max((T + p - 1) / p, kMinQuota);
    if (run <= a.quota + C::kSecondRow) {
      a.quota = run;
      a.pieces = (T + run - 1) / run;
      ctas = rows * a.pieces;
    }
  }
  a.ctas = ctas;
  // A row in many pieces is merged by a kernel with a CTA per head, which costs
  // a launch (about as much as 16 loads in a row) and 4 more a wave of its CTAs, 8
  // to a multiprocessor, instead of by its last CTA: by the loads that a thread of
  // each has in a row.  us, last CTA against kernel, at rows x heads of a row,
  // e4m3: 57K 4x16 73.7, 29.5; 57K 4x8 30.9, 22.2; 4K 8x16 18.8, 12.6; 64K ragged
  // 32x16 86.0, 74.4; 8K ragged 64x16 35.2, 32.8; the other way 4K ragged 128x16
  // 33.3, 36.0; 2K ragged 400x16 47.8, 66.6; 8K 64x4 21.0, 21.7; 128K 16x4 88.4,
  // 89.1; 32K 32x8 51.2, 51.5; 100K 1x1 15.9, 19.3.
  const int pieces = a.pieces > 0 ? a.pieces : (ctas + rows - 1) / rows + 1;
  a.merge_later = pieces * a.G * (D / 4) / (C::W * 32) >
                  pieces * (D / 4) / kMergeThreads + 16 + 4LL * a.B * a.Hq / (num_sms() * 8);
  const sfi_status r = cuda_status(launch_k(k, dim3(ctas), dim3(C::W * 32), C::kSmem, st, a));
  if (r != SFI_OK || !a.merge_later) return r;
  return cuda_status(launch_k(page_merge_kernel<D, LIST>, dim3(a.B * a.Hq), dim3(kMergeThreads), merge_smem(ctas), st, a));
}

template <int D, int FMT, bool LIST>
sfi_status launch_heads(PageAttnArgs& a, cudaStream_t st) {
  if (a.G > 8) return launch<D, FMT, kTwo, LIST>(a, st);
  if (a.G > 4) return launch<D, FMT, kOne, LIST>(a, st);
  return launch<D, FMT, kHalf, LIST>(a, st);
}

template <int FMT, bool LIST>
sfi_status launch_any(int D, PageAttnArgs& a, cudaStream_t st) {
  return D == 128 ? launch_heads<128, FMT, LIST>(a, st) : launch_heads<64, FMT, LIST>(a, st);
}

// Shared by the three entry points: kv (bf16) or q8 (8-bit) is the cache.
sfi_status run(const sfi_shape* shape, const sfi_paged_kv* kv, const sfi_quant_kv* q8, int32_t L, const int32_t* lens,
               const sfi_bf16* q, const int32_t* sel, int32_t sel_ld, int32_t K, bool list, float* out, float* lse,
               void* ws, size_t ws_bytes, sfi_stream stream) {
  SFI_TRY(check_shape(shape));
  SFI_TRY(q8 ? check_quant(q8) : check_kv(kv));
  SFI_TRY(check_L(shape, L));
  if (!q || !aligned16(q) || !out || !aligned16(out)) return SFI_ERR_INVALID_ARG;
  // the kernel loads the pools 32 bytes at a time
  const uintptr_t pools = q8 ? reinterpret_cast<uintptr_t>(q8->k_pool) | reinterpret_cast<uintptr_t>(q8->v_pool)
                             : reinterpret_cast<uintptr_t>(kv->k_pool) | reinterpret_cast<uintptr_t>(kv->v_pool);
  if (pools & 31u) return SFI_ERR_INVALID_ARG;
  if (list) {
    if (!sel) return SFI_ERR_INVALID_ARG;
    if (K < 1 || sel_ld < K) return SFI_ERR_SHAPE;
    if (K > shape->max_pages) return SFI_ERR_SHAPE;
  }
  const long BHl = (long)shape->B * shape->Hkv;
  if (BHl > kMaxRows) return SFI_ERR_UNSUPPORTED;
  const BlockWs w = block_ws(*shape);
  if (!ws || !aligned16(ws) || ws_bytes < w.total) return SFI_ERR_WORKSPACE;
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
  a.scale_log2 = kLog2e / sqrtf((float)shape->D);
  // bits that the tokens a warp can meet take: P up to 2^(bias + kSlack) each
  // stay below 1/2 in all (bf16 pages); tails listed K times, P up to 2^14 for 16
  // tokens each, stay 2^2 below fp32's range (8-bit pages)
  int bits = 0;
  while ((1ll << bits) < (list ? K : 1)) ++bits;
  a.bias = q8 ? kBias : -(float)(bits + 4 + 1) - kSlack;
  a.tail_unit = ldexpf(1.f, 20 + bits);
  a.out = out;
  a.lse = lse;
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + w.part_off);
  a.ml = reinterpret_cast<float*>(static_cast<char*>(ws) + w.ml_off);
  a.arrived = reinterpret_cast<int*>(static_cast<char*>(ws) + w.arrived_off);
  cudaStream_t st = (cudaStream_t)stream;
  const int D = shape->D;
  if (!q8) return launch_any<kBf16, true>(D, a, st);
  if (q8->format == SFI_FMT_E4M3)
    return list ? launch_any<SFI_FMT_E4M3, true>(D, a, st) : launch_any<SFI_FMT_E4M3, false>(D, a, st);
  return list ? launch_any<SFI_FMT_INT8, true>(D, a, st) : launch_any<SFI_FMT_INT8, false>(D, a, st);
}

}  // namespace

// Even runs take at most ceil(total / kMinQuota) CTAs and equal shares of the
// rows at most ceil(T / kMinQuota) each, both at most one wave.
int page_attn_ctas_bound(long long rows, int T) {
  return (int)std::min((long long)num_sms() * kMaxCtas, rows * ((T + kMinQuota - 1) / kMinQuota));
}

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
