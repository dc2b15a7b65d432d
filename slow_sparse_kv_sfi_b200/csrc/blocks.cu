// Block selection: a score for every page ("block" of 16 tokens) of a
// (sequence, KV head) from the int8 bounds of its keys, and the K best.
//
//   u_j = max_h e_h * scale_j * sum_d max(q^_hd hi_jd, q^_hd lo_jd)
//
// Since hi >= lo, the maximum is q^+ . hi + q^- . lo with q^+ = max(q^, 0) and
// q^- = min(q^, 0): one int8 dot product of length 2 D with the page's bounds
// row [hi | lo], for all heads of the group at once on the int8 tensor path
// (m16n8k32: 16 pages x 8 heads).  |sum| <= 127 * 127 * D < 2^21 and the
// scales are powers of two, so u does not depend on the order of the sum: it is
// rounded once, if it lies below 2^-126, and clamped once, if it is too large.
// The two scales must not meet the sum one after the other in fp32 as they are:
// with e_h up to 2^122 and scale_j down to 2^-126 the first product alone can
// leave the range.  So e_h comes in times 2^-16 (the product then lies between
// 2^-142, a multiple of the smallest subnormal, and 2^127, and is exact), and
// the 2^16 goes back in with scale_j (finish_score).
//
// Bound by reading 2 D bytes per (page, KV head).  A thread loads the bytes of
// its fragment straight from global memory: the order of d inside the dot
// product is free as long as q uses the same one, so thread t of a quad takes
// the 16-byte chunks t, t + 4, ... of its two rows.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace sfi {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRow = 16384;       // blocks a row's keys take in one CTA's shared memory (64 KB)
constexpr int kMaxCluster = 8;

struct SelectArgs {
  int B, Hq, Hkv, G, L, num_pages, max_pages, nb;
  int n_sink, n_recent, K;
  const int32_t* lens;
  const __nv_bfloat16* q;
  const int8_t* bounds;
  const float* scale;
  const int32_t* pt;
  float* scores;     // [B * Hkv][ld] (score kernel)
  int64_t ld;
  int32_t* sel;      // [B * Hkv][sel_ld] (select kernel)
  int64_t sel_ld;
  int* err;
};

__device__ __forceinline__ void mma_s8_16832(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr float kScoreUnit = 1.f / 65536.f;

// The score from x = 2^-16 max_h sum * e_h and the page's scale: below 1 the
// scale takes the 2^16 (the product is then rounded once), from 1 on the result
// does (only a score that is too large overflows on the way).  Clamped to the
// finite range; -0 becomes +0, its equal.
__device__ __forceinline__ float finish_score(float x, float scale) {
  const float big = __uint_as_float(0x7f7fffffu), unit = 1.f / kScoreUnit;
  const bool small = scale < 1.f;
  const float u = (x * (small ? scale * unit : scale)) * (small ? 1.f : unit);
  return __fadd_rn(fminf(fmaxf(u, -big), big), 0.f);
}

// The group's query codes, as the B operands of the products ([column tile]
// [16-byte chunk of a thread][lane]), and every head's scale times 2^-16.
template <int D, int NT>
struct Query {
  uint4 b[NT][2 * D / 64][32];
  float e[NT * 8];
};

// Whole CTA.  Chunk c of lane (g, t) holds bytes (t + 4 c) * 16 ... of head
// nt * 8 + g's 2 D codes [max(q^, 0) | min(q^, 0)].
template <int D, int NT>
__device__ __forceinline__ void load_query(const SelectArgs& a, int b, int h, Query<D, NT>& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int n = warp; n < NT * 8; n += kWarps) {
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
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int at = half * D + lane * E + e;           // byte of the head's row of codes
        const int chunk = at / 16, t = chunk % 4, j = chunk / 4;
        reinterpret_cast<int8_t*>(&s.b[n / 8][j][(n % 8) * 4 + t])[at % 16] = (int8_t)(half ? min(c, 0) : max(c, 0));
      }
    }
    if (lane == 0) s.e[n] = __uint_as_float((uint32_t)(ex + 127) << 23) * kScoreUnit;   // down to 2^-142, exact
  }
  __syncthreads();
}

// What lane (g, t) of a warp needs to know of blocks tile * 16 + g and
// tile * 16 + 8 + g: the page whose bounds give the score, or (page < 0) the
// score itself: -infinity past the end and for a bad page table entry,
// +infinity for the blocks that are always taken.
struct Where {
  int page[2];
  float fixed[2];
};
__device__ __forceinline__ Where locate(const SelectArgs& a, int b, int len, int tile, int lane) {
  Where w;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int j = tile * 16 + (lane >> 2) + 8 * r;
    w.page[r] = -1;
    w.fixed[r] = -INFINITY;
    if ((long)j * kPage >= len) continue;
    if (j * kPage < a.n_sink || (j + 1) * kPage > len - a.n_recent) {
      w.fixed[r] = INFINITY;
      continue;
    }
    w.page[r] = __ldg(a.pt + (size_t)b * a.max_pages + j);
    if ((unsigned)w.page[r] >= (unsigned)a.num_pages) {
      latch_error(a.err, SFI_ERR_DEVICE_CHECK, kSiteBlockPage);
      w.page[r] = -1;
    }
  }
  return w;
}

// Scores of U tiles for KV head h, by one warp, all loads first: u[i] of lanes
// with t = 0 is that of block 16 * tile + g, of lanes with t = 1 that of block
// 16 * tile + 8 + g.
template <int D, int NT, int U>
__device__ __forceinline__ void score_tiles(const SelectArgs& a, int h, const Where (&w)[U], int lane,
                                            const Query<D, NT>& s, float (&u)[U]) {
  constexpr int KC = 2 * D / 64;
  const int t = lane & 3;
  uint4 x[U][2][KC];
  float sc[U][2];
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sc[i][r] = 0.f;
#pragma unroll
      for (int c = 0; c < KC; ++c) x[i][r][c] = make_uint4(0, 0, 0, 0);
      if (w[i].page[r] < 0) continue;
      const size_t ph = (size_t)w[i].page[r] * a.Hkv + h;
      const uint4* row = reinterpret_cast<const uint4*>(a.bounds + ph * 2 * D);
#pragma unroll
      for (int c = 0; c < KC; ++c) x[i][r][c] = __ldg(row + t + 4 * c);
      sc[i][r] = __ldg(a.scale + ph);
    }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      int d[4] = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint4 q = s.b[nt][c][lane];
        const uint32_t a0[4] = {x[i][0][c].x, x[i][1][c].x, x[i][0][c].y, x[i][1][c].y};
        const uint32_t a1[4] = {x[i][0][c].z, x[i][1][c].z, x[i][0][c].w, x[i][1][c].w};
        mma_s8_16832(d, a0, q.x, q.y);
        mma_s8_16832(d, a1, q.z, q.w);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = nt * 8 + 2 * t + (j & 1);
        if (n < a.G) best[j >> 1] = fmaxf(best[j >> 1], (float)d[j] * s.e[n]);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
      best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
    }
    const int r = t & 1;   // the lane's own block: selected before the scale comes in
    const float v = finish_score(r ? best[1] : best[0], r ? sc[i][1] : sc[i][0]);
    u[i] = (r ? w[i].page[1] : w[i].page[0]) >= 0 ? v : r ? w[i].fixed[1] : w[i].fixed[0];
  }
}

// Scores of the blocks below n of row (b, h), two tiles at a time, by warp
// `first` of `warps`: put(block, score).  ready() brings the query into s.
template <int D, int NT, class Ready, class Put>
__device__ __forceinline__ void score_row(const SelectArgs& a, int b, int h, int len, int n, int first, int warps,
                                          int lane, const Query<D, NT>& s, Ready ready, Put put) {
  constexpr int U = 2;
  Where w[U];
#pragma unroll
  for (int i = 0; i < U; ++i) w[i] = locate(a, b, len, first + i * warps, lane);
  ready();
  for (int tile = first; tile * 16 < n; tile += U * warps) {
    Where next[U];
#pragma unroll
    for (int i = 0; i < U; ++i) next[i] = locate(a, b, len, tile + (U + i) * warps, lane);
    float u[U];
    score_tiles<D, NT, U>(a, h, w, lane, s, u);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int j = (tile + i * warps) * 16 + (lane >> 2) + 8 * (lane & 1);
      if ((lane & 2) == 0 && j < n) put(j, u[i]);
      w[i] = next[i];
    }
  }
}

// Scores alone, for rows that the select kernel does not hold.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) block_score_kernel(const SelectArgs a) {
  grid_dep_enter();
  __shared__ Query<D, NT> s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.y, b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int len = seq_len(a.lens, a.L, b, a.err);
  float* row = a.scores + (size_t)bh * a.ld;
  score_row<D, NT>(a, b, h, len, a.nb, blockIdx.x * kWarps + warp, gridDim.x * kWarps, lane, s,
                   [&]() { load_query<D, NT>(a, b, h, s); }, [&](int j, float u) { row[j] = u; });
}

// A key back to its score (the inverse of float_key).
__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

constexpr uint32_t kForced = 0xffffffffu;   // key of a block that is always taken (float_key gives less)
constexpr int kBins = 4 * kThreads;

struct Search {
  uint32_t cnt[2][kWarps][4];
  int scan[kWarps];
  int hist[kBins];
  uint32_t cand[kThreads];
  int bin, above, m;
  uint32_t threshold;
};

// The K-th largest of keys[0, n), n > K, by the whole CTA, or any value that
// splits off K keys.  A histogram over kBins equal steps of the score gives the
// bin of the K-th largest; of its few keys each thread ranks one.  A bin that
// holds more than kThreads keys (equal or very uneven scores) is left to a
// bisection over the keys: three thresholds a round, counted by the whole CTA.
__device__ __forceinline__ uint32_t kth_key(const uint32_t* keys, int n, int K, Search& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // forced blocks, smallest and largest other key.  (Rolled loops over shared
  // memory: this code runs once per CTA, so its own size costs most.)
  uint32_t mn = kForced, mx = 0u, forced = 0u;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint32_t k = keys[i];
    forced += k == kForced;
    mn = min(mn, k);
    mx = max(mx, k == kForced ? 0u : k);
  }
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  forced = __reduce_add_sync(0xffffffffu, forced);
  if (lane == 0) *reinterpret_cast<uint4*>(s.cnt[0][warp]) = make_uint4(mn, mx, forced, 0u);
#pragma unroll
  for (int i = 0; i < 4; ++i) s.hist[i * kThreads + threadIdx.x] = 0;
  if (threadIdx.x == 0) s.m = 0;
  __syncthreads();
  // (lane w takes warp w's: kWarps reads by every lane took 500 cycles more)
  const uint4 v = lane < kWarps ? *reinterpret_cast<const uint4*>(s.cnt[0][lane]) : make_uint4(kForced, 0u, 0u, 0u);
  uint32_t lo = __reduce_min_sync(0xffffffffu, v.x);
  uint32_t hi = __reduce_max_sync(0xffffffffu, v.y);
  forced = __reduce_add_sync(0xffffffffu, v.z);
  const int need = K - (int)forced;
  if (need <= 0) return kForced - 1u;   // the forced ones are all
  // monotone in the score; a range that overflows puts all into one bin, and
  // -infinity (a bad page) goes to the lowest
  const float s0 = fmaxf(key_score(lo), -3.402823466e38f);
  const float step = __fdiv_rn((float)kBins, key_score(hi) - s0);
  auto bin_of = [&](uint32_t k) { return max(0, min(kBins - 1, (int)((key_score(k) - s0) * step))); };
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint32_t k = keys[i];
    if (k != kForced) atomicAdd(&s.hist[bin_of(k)], 1);
  }
  __syncthreads();
  // sums from the top: thread t owns bins kBins - 4 t - 1 down to kBins - 4 t - 4
  int bins[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bins[i] = s.hist[kBins - 1 - 4 * (int)threadIdx.x - i];
    sum += bins[i];
  }
  int x = sum;
#pragma unroll
  for (int sh = 1; sh < 32; sh <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, sh);
    if (lane >= sh) x += y;
  }
  if (lane == 31) s.scan[warp] = x;
  __syncthreads();
  int above = x - sum + (int)__reduce_add_sync(0xffffffffu, lane < warp ? (unsigned)s.scan[lane] : 0u);
  if (above < need && above + sum >= need) {   // one thread
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (above < need && above + bins[i] >= need) {
        s.bin = kBins - 1 - 4 * (int)threadIdx.x - i;
        s.above = above;
      }
      above += bins[i];
    }
  }
  __syncthreads();
  const int bin = s.bin;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint32_t k = keys[i];
    if (k != kForced && bin_of(k) == bin) {
      const int at = atomicAdd(&s.m, 1);
      if (at < kThreads) s.cand[at] = k;
    }
  }
  __syncthreads();
  const int m = s.m;
  if (m <= kThreads) {
    const int rank = need - s.above;   // the rank-th largest of the bin
    if ((int)threadIdx.x < m) {
      const uint32_t k = s.cand[threadIdx.x];
      int gt = 0, ge = 0;
      for (int i = 0; i < m; ++i) {
        gt += s.cand[i] > k;
        ge += s.cand[i] >= k;
      }
      if (gt < rank && ge >= rank) s.threshold = k;   // equal keys write the same
    }
    __syncthreads();
    return s.threshold;
  }
  // bisection: at least K keys are >= lo, and at most the forced ones > hi
  for (int round = 1; lo < hi; ++round) {
    const uint32_t d = hi - lo;
    // lo < m0 <= m1 <= m2 <= hi
    const uint32_t m0 = lo + (d >> 2) + 1, m1 = max(m0, lo + (d >> 1) + 1), m2 = max(m1, lo + (d >> 1) + (d >> 2) + 1);
    uint32_t c0 = 0, c1 = 0, c2 = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint32_t k = keys[i];
      c0 += k >= m0;
      c1 += k >= m1;
      c2 += k >= m2;
    }
    c0 = __reduce_add_sync(0xffffffffu, c0);
    c1 = __reduce_add_sync(0xffffffffu, c1);
    c2 = __reduce_add_sync(0xffffffffu, c2);
    if (lane == 0) *reinterpret_cast<uint4*>(s.cnt[round & 1][warp]) = make_uint4(c0, c1, c2, 0u);
    __syncthreads();   // the readers of this buffer's last use are past the last round's barrier
    const uint4 w = lane < kWarps ? *reinterpret_cast<const uint4*>(s.cnt[round & 1][lane]) : make_uint4(0u, 0u, 0u, 0u);
    c0 = __reduce_add_sync(0xffffffffu, w.x);
    c1 = __reduce_add_sync(0xffffffffu, w.y);
    c2 = __reduce_add_sync(0xffffffffu, w.z);
    uint32_t c;
    if (c2 >= (uint32_t)K) {
      lo = m2;
      c = c2;
    } else if (c1 >= (uint32_t)K) {
      lo = m1;
      hi = m2 - 1;
      c = c1;
    } else if (c0 >= (uint32_t)K) {
      lo = m0;
      hi = m1 - 1;
      c = c0;
    } else {
      hi = m0 - 1;
      c = 0;
    }
    if (c == (uint32_t)K) break;   // lo splits off K keys
  }
  return lo;
}

// Scores and selection of one row by a cluster of CTAs: all of them score a
// share of the row's blocks into the first one's shared memory, which then
// finds the K-th largest key and writes the chosen blocks in order.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) block_select_kernel(const SelectArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();   // this CTA runs, so its shared memory may be written
  grid_dep_enter();
  extern __shared__ __align__(16) uint32_t keys[];   // of the cluster's first CTA
  __shared__ union Shared {
    Query<D, NT> query;
    Search search;
  } sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int bh = blockIdx.x / cs, b = bh / a.Hkv, h = bh - b * a.Hkv;
  int32_t* out = a.sel + (size_t)bh * a.sel_ld;
  const int len = seq_len(a.lens, a.L, b, rank == 0 && threadIdx.x == 0 ? a.err : nullptr);
  const int n = (len + kPage - 1) / kPage;
  if (n <= a.K) {   // the same in every CTA of the cluster
    if (rank == 0)
      for (int i = threadIdx.x; i < a.K; i += kThreads) out[i] = i;
    cl.barrier_wait();
    return;
  }
  uint32_t* first = cl.map_shared_rank(keys, 0);
  score_row<D, NT>(a, b, h, len, n, rank * kWarps + warp, cs * kWarps, lane, sh.query,
                   [&]() {
                     load_query<D, NT>(a, b, h, sh.query);
                     cl.barrier_wait();
                   },
                   [&](int j, float u) { first[j] = u == INFINITY ? kForced : float_key(u); });
  cl.sync();
  if (rank != 0) return;
  const uint32_t lo = kth_key(keys, n, a.K, sh.search);
  __syncthreads();   // its shared memory is used again
  int* scan = sh.search.scan;

  // All keys above lo, and the first of those equal to it.  Warp w has the w-th
  // run of positions, lane c the c-th 32 of it as two masks, so the chosen ones
  // come out in order.
  const int run = (n + 32 * kWarps - 1) / (32 * kWarps) * 32;   // at most 1024: 32 times 32
  const int i0 = warp * run;
  uint32_t ma = 0, me = 0;
#pragma unroll 4
  for (int c = 0; c < run / 32; ++c) {
    const int i = i0 + c * 32 + lane;
    const uint32_t k = i < n ? keys[i] : 0u;   // below lo
    const uint32_t x = __ballot_sync(0xffffffffu, k > lo), y = __ballot_sync(0xffffffffu, k == lo);
    if (lane == c) {
      ma = x;
      me = y;
    }
  }
  // both counts in one word: at most 16384 of each
  const int own = __popc(ma) | (__popc(me) << 16);
  int x = own;
#pragma unroll
  for (int sh_ = 1; sh_ < 32; sh_ <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, sh_);
    if (lane >= sh_) x += y;
  }
  if (lane == 31) scan[warp] = x;
  __syncthreads();
  const unsigned of = lane < kWarps ? (unsigned)scan[lane] : 0u;
  const int total = (int)__reduce_add_sync(0xffffffffu, of & 0xffffu);
  const int before = x - own + (int)__reduce_add_sync(0xffffffffu, lane < warp ? of : 0u);
  const int take = a.K - total, eq = before >> 16;   // equal ones to take, and those in front of this lane's
  int at = (before & 0xffff) + min(eq, take);
  for (int drop = __popc(me) - max(take - eq, 0); drop > 0; --drop) me &= ~(0x80000000u >> __clz(me));
  for (uint32_t m = ma | me; m; m &= m - 1) out[at++] = i0 + lane * 32 + __ffs(m) - 1;
}

// A cluster per row: the largest that lets all rows run at once and leaves every
// warp a tile.  A cluster lies inside a GPC, whose multiprocessors it may not
// use up, so the device says how many it holds (one CTA per multiprocessor: 15
// clusters of 7 or 8, 22 of 6, 26 of 5, 33 of 4, 45 of 3, 74 of 2).  us for rows
// of 8193 blocks, clusters of 4, 6, 8: 15 rows 21.5, 18.6, 16.5; 16 rows 22.1,
// 19.1, 24.6; 24 rows 23.9, 32.3, 28.0.
template <int D, int NT>
cudaError_t launch_select(const SelectArgs& a, int BH, cudaStream_t st) {
  auto k = block_select_kernel<D, NT>;
  static DeviceOnce once;
  static std::atomic<int> room[64][kMaxCluster + 1];   // by device and cluster size
  int dev = 0;
  cudaGetDevice(&dev);
  dev &= 63;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  if (!once.done()) {
    cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRow * (int)sizeof(uint32_t));
    cfg.dynamicSmemBytes = kMaxRow * sizeof(uint32_t);
    cfg.numAttrs = 2;
    for (int cs = 1; cs <= kMaxCluster && e == cudaSuccess; ++cs) {
      cfg.gridDim = dim3(cs);
      attr[1].val.clusterDim.x = cs;
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
      room[dev][cs].store(n);
    }
    if (!once.mark(e)) return e;
  }
  int cs = std::min(kMaxCluster, (a.nb + kWarps * 16 - 1) / (kWarps * 16));
  while (cs > 1 && BH > room[dev][cs].load()) --cs;
  cfg.gridDim = dim3(BH * cs);
  cfg.dynamicSmemBytes = (size_t)((a.nb + 3) / 4 * 4) * sizeof(uint32_t);
  cfg.stream = st;
  attr[1].val.clusterDim.x = cs;
  cfg.numAttrs = cs > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace

// The arrival counts come first and have one size: a workspace may then serve
// layers of several shapes, each of which finds them zero.
BlockWs block_ws(const sfi_shape& s) {
  BlockWs w{};
  const long long BH = (long long)s.B * s.Hkv;
  const int G = s.Hq / s.Hkv;
  w.arrived_off = 0;
  size_t off = align_up((size_t)kMaxRows * sizeof(int), 256);
  w.score_off = off;
  off += align_up((size_t)BH * (((size_t)s.max_pages + 3) / 4 * 4) * sizeof(float), 256);
  const size_t items = 2 * (size_t)page_attn_ctas_bound(BH, s.max_pages);
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
  if (nb > topk_max_n() || (long)shape->B * shape->Hkv > kMaxRows) return SFI_ERR_UNSUPPORTED;
  const BlockWs w = block_ws(*shape);
  if (!ws || !aligned16(ws) || ws_bytes < w.total) return SFI_ERR_WORKSPACE;
  const int BH = shape->B * shape->Hkv;
  SelectArgs a{};
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
  a.K = K;
  a.lens = lens;
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.bounds = index->bounds;
  a.scale = index->scale;
  a.pt = index->page_table;
  a.scores = reinterpret_cast<float*>(static_cast<char*>(ws) + w.score_off);
  a.ld = (nb + 3) / 4 * 4;
  a.sel = sel;
  a.sel_ld = sel_ld;
  a.err = index->err;
  cudaStream_t st = (cudaStream_t)stream;
  const bool wide = a.G > 8;
  cudaError_t e;
  if (nb <= kMaxRow) {
    e = shape->D == 128 ? (wide ? launch_select<128, 2>(a, BH, st) : launch_select<128, 1>(a, BH, st))
                        : (wide ? launch_select<64, 2>(a, BH, st) : launch_select<64, 1>(a, BH, st));
  } else {
    const int tiles = (nb + 15) / 16;
    int gx = (tiles + kWarps - 1) / kWarps;
    const int cap = (num_sms() * 4 + BH - 1) / BH;
    if (gx > cap) gx = cap;
    auto k = shape->D == 128 ? (wide ? block_score_kernel<128, 2> : block_score_kernel<128, 1>)
                             : (wide ? block_score_kernel<64, 2> : block_score_kernel<64, 1>);
    e = launch_k(k, dim3(gx, BH), dim3(kThreads), 0, st, a);
  }
  if (e != cudaSuccess || nb <= kMaxRow) return cuda_status(e);
  return run_topk(BH, nb, a.scores, a.ld, K, 0, sel, sel_ld, nullptr, 0, st);
}

}  // extern "C"
