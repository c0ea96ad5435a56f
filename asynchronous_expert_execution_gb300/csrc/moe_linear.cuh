// What the products share (the forward product, its gradients): tiles, kernels and their choice.
//
// Weights are the MMA's 128 (or, over two SMs, 256) rows and tokens its columns, so few tokens and
// thousands run on the same tiles: D[feature, token], tiles of 128 bytes of K by TMA, accumulators in
// TMEM.  The epilogue passes through
// shared memory as [token][feature]: a thread of a TMEM lane writes its feature's column there,
// and reads back 8 adjacent features of one token, so rows move in 16-byte units (storing from
// the lanes directly, 2 bytes a thread, cost 67,000 cycles a 128 x 256 tile, twice the products
// of a 7168-deep e4m3 tile; turning a whole tile's features at once, with two barriers of 128
// threads per 16 tokens, 17,000).
//
//   pair   persistent, tiles of 256 features x up to 256 tokens (128 for fp32 results) over two SMs
//          (cta_group::2): each SM stages half of both operands, which halves the shared-memory traffic per product.
//   split  one tile of 128 features x up to 128 tokens per cluster of up to 8 CTAs, K split over
//          them; partials meet through distributed shared memory in rank order (no workspace,
//          no atomics).  For few tiles: a lone SM streams weights far below the HBM rate.
//
// Every wait is bounded (2 s): a wait that runs out stops all roles, latches MOE_ERR_TIMEOUT in
// the operators' error word, and the CTA still lets what is in flight land and frees its TMEM.
#pragma once
#include <cuda_fp8.h>
#include <cudaTypedefs.h>
#include <algorithm>
#include <atomic>
#include <cmath>
#include "moe_ops.cuh"
#include "moe_ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

__device__ unsigned int g_ops_error;

constexpr int kBM = 128;                           // weight rows per CTA
constexpr int kBKBytes = 128;                      // K of a k-block (one swizzle atom)
constexpr int kABlock = kBM * kBKBytes;            // 16 KB
constexpr int kThreads = 256;                      // warps: TMA, MMA, TMEM, spare, 4 x epilogue
constexpr unsigned long long kLimitNs = 2000000000ull;
// The tensor cores' fp32 sums cut what does not fit, so their error grows with the length of a sum
// (bf16, 7168 deep, of the result's norm: 2.6e-6 in one sum, 1.4e-6 in sums of 22 k-blocks, 7.2e-7 in
// sums of 12, 4.8e-7 in sums of 8; plain fp32 products 2e-7 to 9e-7).  Results that are kept in fp32 are
// therefore summed in chunks of up to this many k-blocks, which the epilogue adds with rounding (2048 x 7168 x
// 7168: 142 us in chunks of 12, 157 in chunks of 8); a bf16 result's own rounding is 1,000 times larger.
constexpr int kChunkBlocks = 12;

// The product, and the two of its gradient with y [T, N] and w [N, F] in the forward product's names:
//   kForward     y[t, n]    = sum_f x[t, f] w[n, f]        both operands K-major
//   kRowsGrad    gx[t, f]   = sum_n gy[t, n] w[n, f]       w lies across K
//   kWeightGrad  gw[n, f]   = sum_t gy[t, n] x[t, f]       both lie across K, K is a group's rows
// Each runs as D[feature, token]: features are what is adjacent in the result (n; f; f), tokens its rows (t; t; n).  An
// operand that lies across K comes as boxes of 64 rows of K x 64 elements, as it lies in memory.
enum Product { kForward, kRowsGrad, kWeightGrad };
constexpr int kBoxRows = 64;                       // rows of K in a k-block of an operand that lies across
constexpr int kBox = kBoxRows * kBKBytes;

// T, N, F: the result's rows and features, and K (kWeightGrad: the rows of all groups)
struct LinearParams {
  const float* bias;
  const float* sx;
  const float* sw;
  const void* mul;
  const void* res;
  void* y;
  const int32_t* offsets;
  int64_t ldmul, ldres, ldy;
  int T, N, F, G, act, nk;
  bool wide;                        // y, mul and residual: 16-byte units
  bool beside;                      // kWeightGrad: runs beside the kernel before it (ops_beside)
  __host__ __device__ bool plain() const { return !mul && !res && act == MOE_ACT_NONE; }
};

// Bounded wait; false once it ran out or another role gave up.
template <Order O = kCta>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  for (int i = 0; i < 4; ++i)
    if (mbar_try<O>(bar, parity)) return true;
  constexpr int kTries = 16;                         // between two looks at the clock, which is slow to read
  const unsigned long long t0 = now_ns();
  while (true) {
    for (int i = 0; i < kTries; ++i)
      if (mbar_try<O>(bar, parity)) return true;
    if (*abort_flag) return false;
    if (now_ns() - t0 > kLimitNs) {
      *abort_flag = 1;
      atomicCAS(&g_ops_error, 0u, (unsigned)MOE_ERR_TIMEOUT);
      return false;
    }
  }
}

// After a wait that ran out, when all roles have stopped: copies, products and their arrivals on barriers may still be under
// way, and must not reach shared memory or TMEM that the next CTA owns.  None of them takes a hundredth of this.
constexpr unsigned long long kSettleNs = 10000000ull;
__device__ __forceinline__ void settle(volatile int* abort_flag) {
  if (threadIdx.x != 0 || !*abort_flag) return;
  const unsigned long long t0 = now_ns();
  while (now_ns() - t0 < kSettleNs) __nanosleep(1000);
}

// Rows [a, b) of group g, clipped to the rows there are.
struct Span {
  int a, n;
};
__device__ __forceinline__ Span group_rows(const LinearParams& p, int g, int total) {
  if (!p.offsets) return {0, total};
  const int a = min(total, max(0, __ldg(p.offsets + g))), b = min(total, max(a, __ldg(p.offsets + g + 1)));
  return {a, b - a};
}

// A CTA's 128 rows of A in k-block kb: features f .. of group g (kWeightGrad: of the rows from row0).
template <int CG, int MODE, bool E4M3>
__device__ __forceinline__ void load_a(uint32_t dst, const CUtensorMap* m, uint32_t bar, int kb, int f, int g, int row0) {
  if constexpr (MODE == kForward) {
    tma_3d<CG>(dst, m, bar, kb * (E4M3 ? kBKBytes : kBKBytes / 2), f, g);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (MODE == kRowsGrad)
        tma_3d<CG>(dst + i * kBox, m, bar, f + 64 * i, kb * kBoxRows, g);
      else
        tma_2d<CG>(dst + i * kBox, m, bar, f + 64 * i, row0 + kb * kBoxRows);
    }
  }
}
// kWeightGrad: `cols` columns (a multiple of 64) of B from column c
template <int CG>
__device__ __forceinline__ void load_across(uint32_t dst, const CUtensorMap* m, uint32_t bar, int kb, int c, int cols, int row0) {
  for (int i = 0; i < cols; i += 64) tma_2d<CG>(dst + i * kBKBytes, m, bar, c + i, row0 + kb * kBoxRows);
}

template <int MODE>
__device__ __forceinline__ uint64_t a_desc(uint32_t saddr) { return MODE == kForward ? operand_desc(saddr) : across_desc(saddr, kBox); }
template <int MODE>
__device__ __forceinline__ uint64_t b_desc(uint32_t saddr) { return MODE == kWeightGrad ? across_desc(saddr, kBox) : operand_desc(saddr); }

// The products of one k-block; `live`: rows of K that it holds (kWeightGrad: 16 a product, those behind are left out).
template <int CG, int MODE, bool E4M3>
__device__ __forceinline__ void product_block(uint32_t d, uint32_t smem, uint32_t idesc, bool accumulate, int live) {
  const uint64_t a = a_desc<MODE>(smem), b = b_desc<MODE>(smem + kABlock);
  if (MODE == kWeightGrad && live <= kBoxRows - 16) {
    for (int i = 0; 16 * i < live; ++i) mma<CG, E4M3>(d, a + 128 * i, b + 128 * i, idesc, accumulate || i > 0);
  } else {
    mma_block<CG, E4M3, MODE != kForward, MODE == kWeightGrad>(d, a, b, idesc, accumulate);
  }
}

// kWeightGrad in one CTA, by a whole warp: the last k-block of a group holds `live` rows of it, and behind them rows of the next
// group or of none, with any content.  Those that a product of 16 rows would still reach become zeros in both operands.
__device__ __forceinline__ void clear_rows(uint8_t* stage, int boxes, int live) {
  // a row's eight units of 16 bytes by adjacent lanes, four rows at a time; no divisions: the products wait for this
  const int lane = threadIdx.x % 32, end = (live + 15) / 16 * 16;
  for (int r = live + lane / 8; r < end; r += 4)
    for (int b = 0; b < boxes; ++b) *reinterpret_cast<uint4*>(stage + b * kBox + r * kBKBytes + lane % 8 * 16) = make_uint4(0, 0, 0, 0);
  fence_async();
  __syncwarp();
}

// The tiles of all groups, where a group of n rows has tiles(n), looked up by a whole warp.  64 groups' offsets are
// asked for at a time (1024 groups of 512 x 512 on 8192 rows: 203 us; 32 at a time 211, 128 201, but 32 groups of
// 2880 x 2880 138 / 138 / 140).
struct GroupTiles {
  int g0 = -32, incl = 0;           // 32 groups, and their tiles up to this lane's
  Span sp{0, 0};                    // this lane's group
  int want;                         // the next tile, counted from these groups' first
  __device__ __forceinline__ explicit GroupTiles(int first) : want(first) {}

  // false: there are fewer tiles; then `want` counts from behind the last one
  template <class Tiles>
  __device__ __forceinline__ bool find(const LinearParams& p, Tiles tiles) {
    if (__any_sync(0xffffffffu, want < incl)) return true;
    want -= __shfl_sync(0xffffffffu, incl, 31);
    constexpr int kAt = 2;
    const int lane = threadIdx.x % 32;
    for (int at = g0 + 32; at < p.G; at += 32 * kAt) {
      Span got[kAt];
#pragma unroll
      for (int u = 0; u < kAt; ++u) got[u] = at + 32 * u + lane < p.G ? group_rows(p, at + 32 * u + lane, p.T) : Span{0, 0};
#pragma unroll
      for (int u = 0; u < kAt; ++u) {
        incl = tiles(got[u].n);
        const int all = __reduce_add_sync(0xffffffffu, incl);
        if (want < all) {
          g0 = at + 32 * u;
          sp = got[u];
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
          }
          return true;
        }
        want -= all;
      }
    }
    g0 = -32;
    incl = 0;
    return false;
  }
  // after find: the tile's group, that group's rows, and the tile's number in it
  template <class Tiles>
  __device__ __forceinline__ int get(Tiles tiles, int& g, int& row0, int& n) const {
    const int src = __ffs(__ballot_sync(0xffffffffu, want < incl)) - 1;
    g = g0 + src;
    row0 = __shfl_sync(0xffffffffu, sp.a, src);
    n = __shfl_sync(0xffffffffu, sp.n, src);
    return want - (__shfl_sync(0xffffffffu, incl, src) - tiles(n));
  }
};

// A thread's place in the epilogue's operands: token row r, feature f.
template <typename TO>
struct Place {
  const float* sx;
  const TO* mul;
  const TO* res;
  TO* y;
  __device__ __forceinline__ Place(const LinearParams& p, long long r, int f)
      : sx(p.sx + r), mul(static_cast<const TO*>(p.mul) + r * p.ldmul + f),
        res(static_cast<const TO*>(p.res) + r * p.ldres + f), y(static_cast<TO*>(p.y) + r * p.ldy + f) {}
};

// x / (1 + e^-x), written with e^-|x| so that nothing overflows on the way.  For fp32 results within 10 u (u = 2^-24: the
// exponential and the quotient 4 u each); for bf16 results the fast exponential's 2 + 1.173 |x| steps move it by
// at most 2^-16, 1/256 of their own rounding (4096 x 512 x 7168 with mul, cold caches: bf16 61 us, fp32 80, 75 with the
// fast exponential).
template <typename TO>
__device__ __forceinline__ float silu(float x) {
  const float e = sizeof(TO) == 4 ? expf(-fabsf(x)) : __expf(-fabsf(x));
  return __fdividef(x < 0.f ? x * e : x, 1.0f + e);
}

// x times the normal distribution's integral up to x.  1 + erf of a large negative number cancels (at -5 a tenth of the result
// is lost), so the tail is taken itself: 0.5 erfc(a / sqrt 2) = e^(-a^2 / 2) q(a) for a = |x|, where q falls slowly from 0.5
// to 1 / (a sqrt(2 pi)).  q = t P(t), t = 1 / (1 + 0.35 a): P is a least-squares fit in 64 bits, reweighted until its
// errors are level, and q's relative error stays below 0.6 u on [0, 14.5], past which the result is below fp32.  The
// square's rounding is put back to first order, and fp32 results are within 20 u; for bf16 results neither that nor the
// fast exponential shows (2^-15 together).  4096 x 512 x 7168 with mul, cold caches: bf16
// 78 us, fp32 96; by 1 + erf 78 and 88, by erfc of the whole argument 103 and 120.
// The integral itself; `density`: e^(-x^2 / 2).
template <typename TO>
__device__ __forceinline__ float normal_cdf(float x, float& density) {
  const float a = fminf(fabsf(x), 16.f), s = a * a;
  const float t = __fdividef(1.0f, fmaf(0.35f, a, 1.0f));
  float p = -0.0291578844f;
  p = fmaf(p, t, 0.144030929f);
  p = fmaf(p, t, -0.25583902f);
  p = fmaf(p, t, 0.159319729f);
  p = fmaf(p, t, -0.0232123677f);
  p = fmaf(p, t, 0.105552509f);
  p = fmaf(p, t, 0.119821288f);
  p = fmaf(p, t, 0.139863506f);
  p = fmaf(p, t, 0.139621302f);
  float e;
  if constexpr (sizeof(TO) == 4) {
    e = expf(-0.5f * s);
    e = fmaf(-0.5f * fmaf(a, a, -s), e, e);
  } else {
    e = __expf(-0.5f * s);
  }
  density = e;
  const float tail = e * (p * t);
  return x < 0.f ? tail : 1.0f - tail;
}
template <typename TO>
__device__ __forceinline__ float gelu(float x) {
  float density;
  return x * normal_cdf<TO>(x, density);
}

// The end of the epilogue for one thread, which owns C features of every token it meets: first,
// first + step, ...  C = 8, step = 1: rows of y, mul and residual move in 16-byte units; else
// element by element.  Pointers are to a token's row at feature `first`.  PLAIN: no mul, residual and activation (their tests
// and loads cost a fifth of 4096 x 512 x 7168: 39.4 us, now 32.5).
template <typename TO, int C, bool SCALED, bool PLAIN = false>
struct Finish {
  static constexpr bool kWide = C == 8;
  static constexpr int kVecs = kWide ? C / Vec<TO>::N : C;
  using RV = RowVec<TO, kWide ? Vec<TO>::N : 1>;
  using Raw = typename RV::Raw;
  const LinearParams& p;
  int step, live;                   // live: how many of the C features exist (wide: all or none)
  float sw[C], bias[C];

  __device__ Finish(const LinearParams& q, int g, int first, int step_) : p(q), step(step_) {
    live = first >= q.N ? 0 : min(C, (q.N - first + step_ - 1) / step_);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      sw[i] = SCALED && i < live ? __ldg(q.sw + (size_t)g * q.N + first + i * step) : 1.f;
      bias[i] = q.bias && i < live ? __ldg(q.bias + (size_t)g * q.N + first + i * step) : 0.f;
    }
  }
  // what a token's epilogue reads, ahead of use
  struct Ahead {
    Raw m[kVecs], e[kVecs];
    float sx;
  };
  __device__ __forceinline__ bool on(int i) const { return kWide ? live > 0 : i < live; }
  __device__ __forceinline__ int at(int i) const { return kWide ? i * Vec<TO>::N : i * step; }
  // `token`: whether the token t behind the place's exists
  __device__ __forceinline__ void ahead(Ahead& a, const Place<TO>& place, int t, bool token) const {
    if (SCALED) a.sx = token ? __ldg(place.sx + t) : 1.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if (!PLAIN && p.mul && token && on(i)) a.m[i] = RV::load_rw(place.mul + t * p.ldmul + at(i));
      if (!PLAIN && p.res && token && on(i)) a.e[i] = RV::load_rw(place.res + t * p.ldres + at(i));
    }
  }
  // U tokens' values
  template <int U>
  __device__ __forceinline__ void compute(float (&v)[U][C], const Ahead* a) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < C; ++i) v[u][i] = SCALED ? v[u][i] * (a[u].sx * sw[i]) + bias[i] : v[u][i] + bias[i];
    if (!PLAIN && p.act != MOE_ACT_NONE) {
      auto each_value = [&](auto f) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < C; ++i) v[u][i] = f(v[u][i]);
      };
      if (p.act == MOE_ACT_SILU)
        each_value([](float x) { return silu<TO>(x); });
      else if (p.act == MOE_ACT_GELU)
        each_value([](float x) { return gelu<TO>(x); });
      else
        each_value([](float x) { return x < 0.f ? 0.f : x; });                  // relu; NaN stays
    }
    constexpr int N = C / kVecs;
    auto with = [&](auto raw, auto f) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          float t[N];
          RV::unpack(raw(a[u])[i], t);
#pragma unroll
          for (int j = 0; j < N; ++j) v[u][i * N + j] = f(v[u][i * N + j], t[j]);
        }
    };
    if (!PLAIN && p.mul) with([](const Ahead& h) -> const Raw(&)[kVecs] { return h.m; }, [](float x, float t) { return x * t; });
    if (!PLAIN && p.res) with([](const Ahead& h) -> const Raw(&)[kVecs] { return h.e; }, [](float x, float t) { return x + t; });
  }
  __device__ __forceinline__ void store(const float (&v)[C], TO* y) const {
    constexpr int N = C / kVecs;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float o[N];
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] = v[i * N + j];
      if (on(i)) RV::store(y + at(i), RV::pack(o));
    }
  }
  __device__ __forceinline__ void operator()(float (&v)[C], TO* y, const Ahead& a) const {
    compute(reinterpret_cast<float(&)[1][C]>(v), &a);
    store(v, y);
  }
};

// ------------------------------------------------------------------ split kernel

struct SplitParams {
  CUtensorMap w, x;                 // x: boxes of bn rows
  LinearParams l;
  int bn, stages, splits, nft, ntt; // tokens a tile, ring depth, CTAs a cluster, feature tiles; kWeightGrad: token tiles a group
};

constexpr int kSplitSmem = 226 * 1024;              // of an SM: for one CTA or two

struct SplitTail {                  // behind the stages
  static constexpr int kMaxStages = 12;
  uint64_t full[kMaxStages], empty[kMaxStages], done, got;
  uint32_t tmem;
  int abort_flag;
  int g, row0, nj;                  // this cluster's tile; nj = 0: none
};

// Tokens j0 + tk, + tks, .. < j1 of a tile at features f, f + step, ..: the ranks' partials summed in rank
// order.  This rank's own lie at own [token][128], rank r's share for it at got + r * share [token - j0][128].
template <typename TO, int C, bool SCALED>
__device__ __forceinline__ void split_finish(const SplitParams& p, int g, long long row0, int f0, const float* own, const float* got,
                                             int rank, int j0, int j1, int f, int step, int tk, int tks) {
  constexpr int kAt = C < 8 ? 4 : sizeof(TO) == 2 ? 2 : 1;              // tokens whose mul and residual are in flight
  const Finish<TO, C, SCALED> finish(p.l, g, f0 + f, step);
  const Place<TO> place(p.l, row0 + j0, f0 + f);
  const int share = (j1 - j0) * kBM;
  for (int jb = tk; jb < j1 - j0; jb += kAt * tks) {
    typename Finish<TO, C, SCALED>::Ahead a[kAt];
#pragma unroll
    for (int u = 0; u < kAt; ++u) finish.ahead(a[u], place, jb + u * tks, jb + u * tks < j1 - j0);
    float v[kAt][C];
#pragma unroll
    for (int u = 0; u < kAt; ++u) {
      const int j = min(jb + u * tks, j1 - j0 - 1);
      for (int r = 0; r < p.splits; ++r) {
        const float* from = (r == rank ? own + j0 * kBM : got + r * share) + j * kBM + f;
        float t[C];
        if constexpr (C == 8) {
          const float4 x = *reinterpret_cast<const float4*>(from), y = *reinterpret_cast<const float4*>(from + 4);
          t[0] = x.x, t[1] = x.y, t[2] = x.z, t[3] = x.w, t[4] = y.x, t[5] = y.y, t[6] = y.z, t[7] = y.w;
        } else {
#pragma unroll
          for (int i = 0; i < C; ++i) t[i] = from[step * i];
        }
#pragma unroll
        for (int i = 0; i < C; ++i) v[u][i] = r ? v[u][i] + t[i] : t[i];
      }
    }
    finish.compute(v, a);
#pragma unroll
    for (int u = 0; u < kAt; ++u)
      if (jb + u * tks < j1 - j0) finish.store(v[u], place.y + (jb + u * tks) * p.l.ldy);
  }
}

template <bool E4M3, typename TO, int MODE = kForward>
__global__ void __launch_bounds__(kThreads, 2) linear_split_kernel(const __grid_constant__ SplitParams p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = kABlock + p.bn * kBKBytes;
  SplitTail* s = reinterpret_cast<SplitTail*>(smem + p.stages * stage_bytes);
  volatile int* abort_flag = &s->abort_flag;
  const LinearParams& l = p.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.splits > 1 ? (int)cluster_rank() : 0;
  const int tile = blockIdx.x / p.splits;
  // fp32 results: K in up to four chunks with an accumulator each (see kChunkBlocks)
  constexpr int kAccs = sizeof(TO) == 4 ? 4 : 1;
  const uint32_t cols = max(32, kAccs * p.bn);

  if (threadIdx.x == 0) {
    prefetch_map(&p.w);
    prefetch_map(&p.x);
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&s->full[i], 1);
      mbar_init(&s->empty[i], 1);
    }
    mbar_init(&s->done, 1);
    mbar_init(&s->got, 1);
    s->abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc<1>(&s->tmem, cols);
  int g = 0, nj = 0, row0 = tile / p.nft * p.bn;
  const int fti = tile % p.nft;
  Span sum{0, 0};                                    // kWeightGrad: the group's rows
  if (MODE == kWeightGrad) {
    g = tile / p.nft / p.ntt;
    row0 = tile / p.nft % p.ntt * p.bn;
    nj = min(p.bn, l.T - row0);
    if (l.beside) ops_beside();
    else ops_begin();
    sum = group_rows(l, g, l.F);
    if (sum.n == 0 && l.res) nj = 0;                 // nothing to add
    tc_before();
    __syncthreads();
    tc_after();
  } else if (!l.offsets) {                                  // dense: the tile is known before the inputs are
    nj = min(p.bn, l.T - row0);
    tc_before();
    __syncthreads();
    tc_after();
    ops_begin();
  } else {
    ops_begin();
    if (warp == 3) {                                 // token tile tile / nft of the groups' tiles
      const auto tiles = [&](int n) { return (n + p.bn - 1) / p.bn; };
      GroupTiles at(tile / p.nft);
      if (at.find(l, tiles)) {
        int n;
        const int t = at.get(tiles, g, row0, n);
        row0 += t * p.bn;
        nj = min(p.bn, n - t * p.bn);
      }
      if (lane == 0) {
        s->g = g;
        s->row0 = row0;
        s->nj = nj;
      }
    }
    tc_before();
    __syncthreads();
    tc_after();
    g = s->g;
    row0 = s->row0;
    nj = s->nj;
  }
  const uint32_t tmem = s->tmem;
  const int nk = MODE == kWeightGrad ? (sum.n + kBoxRows - 1) / kBoxRows : l.nk;
  const int kb0 = (int)((long long)nk * rank / p.splits), kb1 = (int)((long long)nk * (rank + 1) / p.splits);
  constexpr int kElems = E4M3 ? kBKBytes : kBKBytes / 2;
  const int chunks = min(kAccs, (kb1 - kb0 + kChunkBlocks - 1) / kChunkBlocks);

  if (nj > 0 && warp == 0 && elect()) {
    uint32_t st = 0, phase = 1;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!wait(&s->empty[st], phase, abort_flag)) break;
      const uint32_t a = smem_u32(smem + st * stage_bytes);
      mbar_expect(&s->full[st], stage_bytes);
      load_a<1, MODE, E4M3>(a, &p.w, smem_u32(&s->full[st]), kb, fti * kBM, g, sum.a);
      if constexpr (MODE == kWeightGrad)
        load_across<1>(a + kABlock, &p.x, smem_u32(&s->full[st]), kb, row0, p.bn, sum.a);
      else
        tma_2d<1>(a + kABlock, &p.x, smem_u32(&s->full[st]), kb * kElems, row0);
      if (++st == p.stages) st = 0, phase ^= 1;
    }
  } else if (MODE == kWeightGrad && nj > 0 && warp == 1) {
    const uint32_t idesc = mma_desc<E4M3, true, true>(kBM, p.bn);
    // this rank's k-blocks; the group's last one, if it is not full, by the whole warp, which clears what lies behind the end
    const int live = sum.n - (nk - 1) * kBoxRows, last = kb1 == nk && kb1 > kb0 && live < kBoxRows ? 1 : 0;
    bool ok = true;
    uint32_t st = 0, phase = 0;
    int chunk = 0, i = 0;                            // block i of the chunk
    const auto block = [&](int rows) {
      uint8_t* stage = smem + st * stage_bytes;
      tc_after();
      product_block<1, MODE, E4M3>(tmem + chunk * p.bn, smem_u32(stage), idesc, i > 0, rows);
      commit<1>(&s->empty[st]);
    };
    const auto next = [&] {
      if (++st == p.stages) st = 0, phase ^= 1;
      if (++i == (kb1 - kb0) * (chunk + 1) / chunks - (kb1 - kb0) * chunk / chunks) ++chunk, i = 0;
    };
    if (elect()) {
      for (int kb = kb0; kb < kb1 - last; ++kb) {
        if (!(ok = wait(&s->full[st], phase, abort_flag))) break;
        block(kBoxRows);
        next();
      }
      if (ok && !last) commit<1>(&s->done);
    }
    __syncwarp();
    if (last) {
      const int src = __ffs(__ballot_sync(0xffffffffu, i > 0 || chunk > 0 || st > 0)) - 1;      // the lane that issued, if one did
      if (src >= 0) {
        st = __shfl_sync(0xffffffffu, st, src), phase = __shfl_sync(0xffffffffu, phase, src);
        chunk = __shfl_sync(0xffffffffu, chunk, src), i = __shfl_sync(0xffffffffu, i, src);
      }
      if (__all_sync(0xffffffffu, ok) && __all_sync(0xffffffffu, wait(&s->full[st], phase, abort_flag))) {
        if (live % 16) clear_rows(smem + st * stage_bytes, 2 + p.bn / 64, live);
        if (elect()) {
          block(live);
          commit<1>(&s->done);
        }
      }
    }
  } else if (nj > 0 && warp == 1 && elect()) {
    const uint32_t idesc = mma_desc<E4M3, MODE != kForward>(kBM, p.bn);
    bool ok = true;
    uint32_t st = 0, phase = 0;
    for (int chunk = 0; chunk < chunks && ok; ++chunk) {
      const int n = (kb1 - kb0) * (chunk + 1) / chunks - (kb1 - kb0) * chunk / chunks;
      for (int i = 0; i < n; ++i) {
        if (!(ok = wait(&s->full[st], phase, abort_flag))) break;
        tc_after();
        product_block<1, MODE, E4M3>(tmem + chunk * p.bn, smem_u32(smem + st * stage_bytes), idesc, i > 0, kBoxRows);
        commit<1>(&s->empty[st]);
        if (++st == p.stages) st = 0, phase ^= 1;
      }
    }
    if (ok) commit<1>(&s->done);
  }
  float* own = reinterpret_cast<float*>(smem);       // [token][feature]: the ring is idle by then
  float* got = own + p.bn * kBM;                     // the other ranks' partials of this rank's share
  const int j0 = nj * rank / p.splits, j1 = nj * (rank + 1) / p.splits;
  if (nj > 0 && warp >= 4) {
    const int q = warp & 3, row = 32 * q + lane;     // TMEM lane: a feature
    const bool ok = __all_sync(0xffffffffu, wait(&s->done, 0, abort_flag));      // whole warps read TMEM
    tc_after();
    if (ok) {
      const uint32_t t = tmem + ((uint32_t)(32 * q) << 16);
      for (int c = 0; c < nj; c += 16) {
        float v[16] = {};
        if (MODE != kWeightGrad || chunks > 0) tmem_ld16(t + c, v);                // no rows: zeros
        for (int ch = 1; ch < chunks; ++ch) {
          float o[16];
          tmem_ld16(t + ch * p.bn + c, o);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] += o[j];
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) own[(c + j) * kBM + row] = v[j];
      }
    }
    if (p.splits > 1) fence_async();
    if (p.splits > 1 && threadIdx.x == 128) mbar_expect(&s->got, (p.splits - 1) * (j1 - j0) * kBM * 4);
  }
  __syncwarp();
  if (p.splits > 1) {
    // every share goes to its rank by bulk copies (reading the ranks' memory by loads moved 1.9 TB/s
    // over the GPU: 9 us for 8 partials of 128 x 128)
    cluster_sync();                                  // all rings are idle, all partials written
    if (nj > 0 && warp == 0 && lane < p.splits && lane != rank) {
      const int i0 = nj * lane / p.splits, i1 = nj * (lane + 1) / p.splits, share = (i1 - i0) * kBM;
      if (share > 0)
        bulk_to_cluster(mapa(smem_u32(got + rank * share), lane), smem_u32(own + i0 * kBM), share * 4,
                        mapa(smem_u32(&s->got), lane));
    }
    if (nj > 0) wait<kCluster>(&s->got, 0, abort_flag);
  } else {
    __syncthreads();
  }
  const long long yrow = MODE == kWeightGrad ? (long long)g * l.T + row0 : row0;
  if (nj > 0) {                                      // every rank sums and finishes its share of the tokens
    if (l.wide)
      split_finish<TO, 8, E4M3>(p, g, yrow, fti * kBM, own, got, rank, j0, j1, threadIdx.x % 16 * 8, 1, threadIdx.x / 16, kThreads / 16);
    else
      split_finish<TO, 4, E4M3>(p, g, yrow, fti * kBM, own, got, rank, j0, j1, lane, 32, warp, kThreads / 32);
  }
  settle(abort_flag);
  if (p.splits > 1) cluster_sync();                  // the copies out of a rank's memory have been received
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 2) tmem_dealloc<1>(tmem, cols);
  if (MODE == kWeightGrad && l.beside) ops_end_beside();
}

// ------------------------------------------------------------------ pair kernel

// tokens of a tile: two accumulators of 256 columns, or three of 128 that take the chunks of fp32 sums in
// turn and 128 columns for the chunks' sum
template <typename TO> constexpr int kPairTokens = sizeof(TO) == 4 ? 128 : 256;
constexpr int kPairRing = 192 * 1024;
constexpr int kPairThreads = 384;                    // warps: TMA, MMA, TMEM, spare, 2 x 4 epilogue
constexpr int kChunk = 32;                           // tokens an epilogue warp turns at a time
constexpr int kTurn = kChunk * 32;                   // floats: 32 tokens x 32 features
constexpr int kStaging = 8 * kTurn * 4;
// kWeightGrad: half a tile's tokens for 32 features a warp, which leave in one box
constexpr int kBoxStaging = 2 * kStaging;
constexpr int pair_ring(int mode) { return mode == kWeightGrad ? kPairRing + kStaging - kBoxStaging : kPairRing; }
template <typename TO> constexpr int kBoxTokens = kPairTokens<TO> / 2;
static_assert(kBoxTokens<float> * 32 * 4 * 8 == kBoxStaging && kBoxTokens<__nv_bfloat16> * 32 * 2 * 8 == kBoxStaging, "a box a warp");

// Quotients by a number that the host knows: a division takes some 120 cycles, and every role of a CTA walks its tiles by itself.
struct Divide {
  uint32_t d, magic;                // floor(2^32 / d) + 1: exact while n d < 2^32; 0: d is one, or not small enough
  static Divide by(int64_t d, int64_t most) { return {(uint32_t)d, d > 1 && d * most < (1ll << 32) ? (uint32_t)((1ll << 32) / d + 1) : 0}; }
  __device__ __forceinline__ int operator()(int n) const { return magic ? (int)__umulhi((uint32_t)n, magic) : n / (int)d; }
};

struct PairParams {
  CUtensorMap w, x[4];              // x: boxes of 16, 32, 64 and tokens / 2 rows; kWeightGrad: 64 rows of K
  LinearParams l;
  CUtensorMap y;                    // kWeightGrad, boxed: the result, boxes of half a tile's rows x 32 features
  bool boxed;
  Divide by_band, by_last;          // kWeightGrad: eight token tiles' feature tiles; the token tiles behind the last eight
  int nft, ntt;                     // feature tiles of 256; kWeightGrad: token tiles a group
  int tokens;                       // of a tile, a multiple of 32
  int stages, stage_bytes;          // of the ring: a k-block of a full tile each
};

// kWeightGrad per expert: how a group's last k-block comes (load_end), of w and of x: windows of 64 rows, boxes of 16 rows and of one.
struct AcrossParams : PairParams {
  CUtensorMap window[2], slab[2], row[2];
};
template <int MODE> using PairArgs = std::conditional_t<MODE == kWeightGrad, AcrossParams, PairParams>;

// kWeightGrad over two CTAs: the last `live` rows of a group, from `row` on, where `live` is no multiple of 16 and less than 64.  Behind them lie
// rows of the next group or of none, with any content, of which products of 16 rows would still reach some; so copies have to bring zeros
// there, and all of a pair's operands come by copies that its leader waits for.  (One box, and a warp of either CTA that clears the rows
// behind the end and tells the leader, wants a release over the cluster, which waits for all that the thread has under way: 32 experts
// 8192 x 2880 x 2880 took 287 us in fp32, here 243; in boxes of 1, 2, 4 .. rows and of zeros 307, for a copy takes 60 cycles.)
// A window is 64 rows that end with the group's last one; the box begins 64 - live rows into it, and what lies behind it is zeros.  A
// group that ends within the matrix's first 64 rows has none: boxes of 16 rows, then of one, and of one row of zeros, which lies beside the
// matrix.  (No box begins before the matrix: a window entered ahead of its first row, with the zeros in front, once faulted.)
__device__ __forceinline__ bool has_window(int row, int live) { return row + live >= kBoxRows; }
__device__ __forceinline__ int end_bytes(int row, int live, int cols) {          // of both CTAs
  return 2 * (has_window(row, live) ? kBoxRows : (live + 15) / 16 * 16) * kBKBytes * (2 + cols / 64);
}
__device__ __forceinline__ void load_window(uint32_t dst, const CUtensorMap* windows, uint32_t bar, int c, int cols, int row, int live) {
#pragma unroll 2
  for (int i = 0; i < cols; i += 64) tma_3d<2>(dst + i * kBKBytes, windows, bar, c + i, kBoxRows - live, row + live - kBoxRows);
}
__device__ __forceinline__ void load_rows(uint32_t dst, const AcrossParams& p, int operand, uint32_t bar, int c, int cols, int width, int row, int live) {
  for (int i = 0; i < cols; i += 64) {
    const uint32_t to = dst + i * kBKBytes;
    int r = 0;
    for (; r + 16 <= live; r += 16) tma_2d<2>(to + r * kBKBytes, &p.slab[operand], bar, c + i, row + r);
    for (; r < live; ++r) tma_2d<2>(to + r * kBKBytes, &p.row[operand], bar, c + i, row + r);
    for (; r % 16; ++r) tma_2d<2>(to + r * kBKBytes, &p.row[operand], bar, (width + 7) / 8 * 8, row);
  }
}
__device__ __forceinline__ void load_end(uint32_t dst, const AcrossParams& p, uint32_t bar, int f, int c, int cols, int row, int live) {
  if (has_window(row, live)) {
    load_window(dst, &p.window[0], bar, f, kBM, row, live);
    load_window(dst + kABlock, &p.window[1], bar, c, cols, row, live);
  } else {
    load_rows(dst, p, 0, bar, f, kBM, p.l.N, row, live);
    load_rows(dst + kABlock, p, 1, bar, c, cols, p.l.T, row, live);
  }
}

struct PairTail {
  static constexpr int kMaxStages = 10;
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[4], tempty[4];
  static constexpr int kTold = 4;                    // kWeightGrad: the tiles that a warp tells the others
  uint64_t told[kTold], heard[kTold];
  uint64_t old[8];                  // an epilogue warp's box of what is added to
  int4 tile[kTold][2];
  uint32_t tmem;
  int abort_flag;
  int finishing;                    // tiles whose epilogue has begun
};

struct PairTile {
  int g, row0, nj, fti, nmma, box, brows;   // brows: token rows a CTA stages
  int sum0, sum, nk;                        // kWeightGrad: the rows summed over, from sum0, and their k-blocks; row0 in the group's result
};

// The tiles of a pair of CTAs, in order: every `pairs`-th one.  Every role's warp walks the groups by itself.  Groups
// with a full tile come first, then those with more than half of one: long tiles at the end would leave pairs idle
// (2880 x 2880, 32 groups of 18 to 1151 rows: 138 us, in the groups' order 142; e4m3 88 and 92; 64 groups of 2048 x
// 768 on 16384 rows 66 and 73).
struct PairWalk {
  GroupTiles at;
  int pass = 0;
  __device__ __forceinline__ PairWalk() : at(blockIdx.x / 2) {}

  // kWeightGrad: all groups have the same tiles, and sums of different lengths.  at.g0: the group; at.want: the tile in it.
  __device__ __forceinline__ bool next_weight(const PairParams& p, PairTile& tl) {
    const int ntt = p.ntt, per = ntt * p.nft;
    while (true) {
      const int before = at.g0;
      if (at.g0 < 0) at.g0 = 0;
      for (; at.want >= per; at.want -= per) ++at.g0;
      if (at.g0 >= p.l.G) return false;
      if (at.g0 != before) at.sp = group_rows(p.l, at.g0, p.l.F);
      if (at.sp.n > 0 || !p.l.res) break;
      at.want += gridDim.x / 2;                      // nothing to add
    }
    tl.g = at.g0;
    const int band = p.by_band(at.want), in = at.want - band * 8 * p.nft, width = min(8, ntt - 8 * band);
    tl.fti = width == 8 ? in >> 3 : p.by_last(in);
    tl.row0 = (8 * band + in - tl.fti * width) * p.tokens;
    tl.nj = min(p.tokens, p.l.T - tl.row0);
    tl.nmma = p.tokens;
    tl.brows = p.tokens / 2;
    tl.sum0 = at.sp.a;
    tl.sum = at.sp.n;
    tl.nk = (at.sp.n + kBoxRows - 1) / kBoxRows;
    at.want += gridDim.x / 2;
    return true;
  }

  // by whole warps
  template <int MODE>
  __device__ __forceinline__ bool next(const PairParams& p, PairTile& tl) {
    if constexpr (MODE == kWeightGrad) return next_weight(p, tl);
    int first = 0, n = p.l.T, local = at.want;
    tl.g = 0;
    if (p.l.offsets) {
      const auto tiles = [&](int rows) {
        const bool now = pass == (rows >= p.tokens ? 0 : 2 * rows > p.tokens ? 1 : 2);
        return now ? (rows + p.tokens - 1) / p.tokens * p.nft : 0;
      };
      while (!at.find(p.l, tiles))
        if (++pass > 2) return false;
      local = at.get(tiles, tl.g, first, n);
    }
    const int ntt = (n + p.tokens - 1) / p.tokens;
    if (local >= ntt * p.nft) return false;
    // eight token tiles meet one feature tile before the next: what runs at one time shares operands in L2
    const int band = local / (8 * p.nft);
    local -= band * 8 * p.nft;
    const int width = min(8, ntt - 8 * band);
    tl.fti = local / width;
    const int j0 = (8 * band + local % width) * p.tokens;
    tl.row0 = first + j0;
    tl.nj = min(p.tokens, n - j0);
    tl.nmma = (tl.nj + 31) & ~31;
    const int half = tl.nmma / 2;                    // token rows each CTA stages: a box that holds them
    tl.box = half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : 3;
    if (16 << tl.box >= p.tokens / 2) tl.box = 3;
    tl.brows = tl.box < 3 ? 16 << tl.box : p.tokens / 2;
    at.want += gridDim.x / 2;
    return true;
  }
};

// The end of a tile's epilogue for one warp, which has 32 features from f on and every other block of 32 of the tile's nj
// tokens, from block `half` on: blocks(body) brings each block's sums into `turn` and calls body(its place - half's).  false: a wait
// ran out there.
// AHEAD: units of mul and residual asked for ahead, where the registers are another's (0: as many as pay).
template <typename TO, bool SCALED, int AHEAD = 0, class Row, class Blocks>
__device__ __forceinline__ bool pair_finish(const LinearParams& l, int g, Row first_row, int f, int nj, int half, const float* turn, Blocks blocks) {
  constexpr bool kSums = sizeof(TO) == 4;
  constexpr int kStep = 2 * kChunk;
  const int lane = threadIdx.x & 31;
  const auto wide = [&](auto plain) {
    constexpr bool PLAIN = decltype(plain)::value;
    // 32 features x 32 tokens turned in the warp's own shared memory: lane i then holds 8
    // features (i % 4) of tokens i / 4 + 8 u, u < 4.  16-byte chunks of a token's row lie at
    // chunk ^ (token & 7): neither the writes nor the reads meet a bank twice.  mul and
    // residual are asked for kAt units ahead, the first ones before the products are done.
    constexpr int kAt = AHEAD ? AHEAD : kSums ? 2 : 4, kU = PLAIN && kAt > 1 ? 2 : 1;         // kU units at once: more would delay the next loads
    const int f8 = lane % 4, tk = lane / 4;
    const Finish<TO, 8, SCALED, PLAIN> finish(l, g, f + f8 * 8, 1);
    const Place<TO> place(l, first_row + half * kChunk + tk, f + f8 * 8);
    const int mine = nj - half * kChunk - tk;           // tokens from this lane's first to the tile's end
    typename Finish<TO, 8, SCALED, PLAIN>::Ahead a[kAt];
#pragma unroll
    for (int u = 0; u < kAt; ++u) finish.ahead(a[u], place, 8 * u, 8 * u < mine);
    return blocks([&](int c) {
#pragma unroll
      for (int u0 = 0; u0 < 4; u0 += kU) {
        float w[kU][8];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const float* row = turn + (tk + 8 * (u0 + u)) * 32;
          const float4 x = *reinterpret_cast<const float4*>(row + ((2 * f8) ^ tk) * 4);
          const float4 y = *reinterpret_cast<const float4*>(row + ((2 * f8 + 1) ^ tk) * 4);
          w[u][0] = x.x, w[u][1] = x.y, w[u][2] = x.z, w[u][3] = x.w, w[u][4] = y.x, w[u][5] = y.y, w[u][6] = y.z, w[u][7] = y.w;
        }
        finish.compute(w, a + u0 % kAt);
#pragma unroll
        for (int u = u0; u < u0 + kU; ++u) {
          if (c + 8 * u < mine) finish.store(w[u - u0], place.y + (c + 8 * u) * l.ldy);
          const int nx = u + kAt < 4 ? c + 8 * (u + kAt) : c + kStep + 8 * (u + kAt - 4);
          finish.ahead(a[u % kAt], place, nx, nx < mine);
        }
      }
    });
  };
  if (l.wide) {
    return l.plain() ? wide(std::true_type{}) : wide(std::false_type{});
  } else {
    // a lane keeps its feature: 32 adjacent elements of a token a warp, kAt tokens at once
    const auto narrow = [&](auto plain) {
      constexpr bool PLAIN = decltype(plain)::value;
      constexpr int kAt = AHEAD ? (kSums ? AHEAD : 2 * AHEAD) : kSums ? PLAIN || SCALED ? 2 : 8 : PLAIN || SCALED ? 8 : 16;
      using F = Finish<TO, 1, SCALED, PLAIN>;
      const F finish(l, g, f + lane, 1);
      const Place<TO> place(l, first_row + half * kChunk, f + lane);
      const int mine = nj - half * kChunk;
      typename F::Ahead a[kAt];
#pragma unroll
      for (int j = 0; j < kAt; ++j) finish.ahead(a[j], place, j, j < mine);
      return blocks([&](int c) {
#pragma unroll 1
        for (int j0 = 0; j0 < kChunk; j0 += kAt) {
          float w[kAt][1];
#pragma unroll
          for (int j = 0; j < kAt; ++j) w[j][0] = turn[(j0 + j) * 32 + (lane ^ (((j0 + j) & 7) << 2))];
          finish.compute(w, a);
          TO* y = place.y + (c + j0) * l.ldy;
#pragma unroll
          for (int j = 0; j < kAt; ++j, y += l.ldy)
            if (c + j0 + j < mine) finish.store(w[j], y);
          const int nx = j0 + kAt < kChunk ? c + j0 + kAt : c + kStep;
#pragma unroll
          for (int j = 0; j < kAt; ++j) finish.ahead(a[j], place, nx + j, nx + j < mine);
        }
      });
    };
    return l.plain() ? narrow(std::true_type{}) : narrow(std::false_type{});
  }
}

template <bool E4M3, typename TO, int MODE = kForward>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ PairArgs<MODE> p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  constexpr bool kAcross = MODE == kWeightGrad;
  constexpr int kRing = pair_ring(MODE);
  PairTail* s = reinterpret_cast<PairTail*>(smem + kPairRing + kStaging);
  volatile int* abort_flag = &s->abort_flag;
  const LinearParams& l = p.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  constexpr int kTokens = kPairTokens<TO>, kAccs = sizeof(TO) == 4 ? 3 : 2;
  constexpr uint32_t kCols = 512;
  const int chunk = sizeof(TO) == 4 ? kChunkBlocks : INT32_MAX; // k-blocks summed in one accumulator

  if (threadIdx.x == 0) {
    prefetch_map(&p.w);
    prefetch_map(&p.x[kAcross ? 0 : 3]);
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&s->full[i], 1);                     // the leader's producer, for both CTAs' bytes
      mbar_init(&s->empty[i], 1);                    // the MMA's commit, in both CTAs
    }
    for (int b = 0; b < kAccs; ++b) {
      mbar_init(&s->tfull[b], 1);
      mbar_init(&s->tempty[b], 16);                  // the epilogue warps of both CTAs, at the leader
    }
    if (kAcross)
      for (int i = 0; i < PairTail::kTold; ++i) {
        mbar_init(&s->told[i], 1);
        mbar_init(&s->heard[i], rank == 0 ? 10 : 9);               // all warps but the telling and the idle ones
      }
    if (kAcross)
      for (int i = 0; i < 8; ++i) mbar_init(&s->old[i], 1);
    s->abort_flag = 0;
    s->finishing = 0;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc<2>(&s->tmem, kCols);
  if (kAcross && l.beside) ops_beside();
  else ops_begin();
  tc_before();
  __syncthreads();
  cluster_sync();
  tc_after();
  const uint32_t tmem = s->tmem;
  PairWalk walk;
  PairTile tl = {};
  constexpr int kElems = E4M3 ? kBKBytes : kBKBytes / 2;
  // The next tile.  kWeightGrad: as a warp tells it, for tiles may be a few k-blocks long and a walk's step takes a role 1,000 cycles.
  uint32_t tiles_heard = 0;
  const auto next_tile = [&]() {
    if constexpr (!kAcross) {
      return walk.template next<MODE>(p, tl);
    } else {
      const int slot = tiles_heard % PairTail::kTold;
      if (!__all_sync(0xffffffffu, wait(&s->told[slot], (tiles_heard / PairTail::kTold) & 1, abort_flag))) return false;
      ++tiles_heard;
      const int4 t = s->tile[slot][0], u = s->tile[slot][1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s->heard[slot]);
      tl.g = t.x, tl.row0 = t.y, tl.nj = t.z, tl.fti = t.w, tl.sum0 = u.x, tl.sum = u.y, tl.nk = u.z;
      tl.nmma = p.tokens, tl.brows = p.tokens / 2;
      return tl.nj > 0;
    }
  };
  // mul and residual of this CTA's i-th tile into L2 while the tile before is finished: the epilogue's 16 KB of
  // reads in flight an SM then last L2's latency (4096 x 512 x 7168 with mul: 50 -> 45 us)
  const auto prefetch = [&](int i) {
    volatile int* finishing = &s->finishing;
    const unsigned long long t0 = now_ns();
    while (!kAcross && *finishing < i && !*abort_flag && now_ns() - t0 < kLimitNs) __nanosleep(200);
    const int f = tl.fti * 2 * kBM + rank * kBM, n = min(kBM, l.N - f) * (int)sizeof(TO), lines = kBM * (int)sizeof(TO) / 128;
    for (int j = lane / lines; j < tl.nj; j += 32 / lines) {
      const int64_t r = (kAcross ? (int64_t)tl.g * l.T : 0) + tl.row0 + j;
      if (lane % lines * 128 < n) {
        if (l.mul) prefetch_l2(reinterpret_cast<const char*>(static_cast<const TO*>(l.mul) + r * l.ldmul + f) + lane % lines * 128);
        if (l.res) prefetch_l2(reinterpret_cast<const char*>(static_cast<const TO*>(l.res) + r * l.ldres + f) + lane % lines * 128);
      }
    }
  };

  if (warp == 0) {
    uint32_t st = 0, phase = 1;
    bool ok = true;
    while (__all_sync(0xffffffffu, ok) && next_tile()) {
      if (!elect()) continue;
      const int wrow = tl.fti * 2 * kBM + rank * kBM, xrow = tl.row0 + rank * (tl.nmma / 2);
      // a group's last rows come by load_end, unless they fill 16s (without groups, copies bring zeros behind the last row by themselves)
      const int nk = kAcross ? tl.nk : l.nk, whole = kAcross && l.offsets && tl.sum % 16 ? nk - 1 : nk;
      for (int kb = 0; kb < nk; ++kb) {
        if (!(ok = wait<kCluster>(&s->empty[st], phase, abort_flag))) break;
        const uint32_t a = smem_u32(smem + st * p.stage_bytes), bar = mapa(smem_u32(&s->full[st]), 0);
        if (!kAcross || kb < whole) {
          if (rank == 0) mbar_expect(&s->full[st], 2 * (kABlock + tl.brows * kBKBytes));
          load_a<2, MODE, E4M3>(a, &p.w, bar, kb, wrow, tl.g, kAcross ? tl.sum0 : 0);
          if constexpr (kAcross)
            load_across<2>(a + kABlock, &p.x[0], bar, kb, xrow, tl.brows, tl.sum0);
          else
            tma_2d<2>(a + kABlock, &p.x[tl.box], bar, kb * kElems, xrow);
        } else if constexpr (kAcross) {
          const int row = tl.sum0 + kb * kBoxRows, live = tl.sum - kb * kBoxRows;
          if (rank == 0) mbar_expect(&s->full[st], end_bytes(row, live, tl.brows));
          load_end(a, p, bar, wrow, xrow, tl.brows, row, live);
        }
        if (++st == p.stages) st = 0, phase ^= 1;
      }
    }
  } else if (kAcross && warp == 3) {
    bool more = true;
    for (uint32_t n = 0; more; ++n) {
      const int slot = n % PairTail::kTold;
      more = walk.template next<MODE>(p, tl);
      if (!__all_sync(0xffffffffu, wait(&s->heard[slot], ((n / PairTail::kTold) & 1) ^ 1, abort_flag))) break;
      if (lane == 0) {
        s->tile[slot][0] = make_int4(tl.g, tl.row0, more ? tl.nj : 0, tl.fti);
        s->tile[slot][1] = make_int4(tl.sum0, tl.sum, tl.nk, 0);
        mbar_arrive(&s->told[slot]);
      }
      __syncwarp();
      if (more && l.res && (sizeof(TO) == 2 || !p.boxed)) prefetch(0);
    }
  } else if (warp == 1 && rank == 0) {
    uint32_t st = 0, phase = 0, acc = 0;
    bool ok = true;
    while (__all_sync(0xffffffffu, ok) && next_tile()) {
      if (!elect()) continue;
      const uint32_t idesc = mma_desc<E4M3, MODE != kForward, kAcross>(2 * kBM, tl.nmma);
      int buf = 0;
      const int nk = kAcross ? tl.nk : l.nk;
      for (int kb = 0, in = chunk; kb < nk; ++kb, ++in) {        // in: k-blocks in this accumulator
        if (in == chunk) {
          if (kb > 0) commit<2>(&s->tfull[buf]);
          buf = acc % kAccs;
          if (!(ok = wait<kTmem>(&s->tempty[buf], ((acc / kAccs) & 1) ^ 1, abort_flag))) break;
          tc_after();
          ++acc;
          in = 0;
        }
        const bool last = kAcross && kb == nk - 1;
        if (!(ok = wait<kCluster>(&s->full[st], phase, abort_flag))) break;
        tc_after();
        product_block<2, MODE, E4M3>(tmem + buf * kTokens, smem_u32(smem + st * p.stage_bytes), idesc, in > 0,
                                     last ? tl.sum - kb * kBoxRows : kBoxRows);
        commit<2>(&s->empty[st]);
        if (++st == p.stages) st = 0, phase ^= 1;
      }
      if (ok && nk > 0) commit<2>(&s->tfull[buf]);
    }
  } else if (warp == 3 && (l.mul || l.res)) {
    for (int i = 0; next_tile(); ++i) prefetch(i);
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp >> 2) - 1;  // TMEM lanes 32 q ..; two warps share a quarter's columns
    float* turn = reinterpret_cast<float*>(smem + kRing + (warp - 4) * (kAcross ? kBoxStaging / 8 : kTurn * 4));
    uint32_t acc = 0, olds = 0;
    // a warp's tokens: every other block of 32, or for boxes the tile's first or second half
    constexpr bool kSums = sizeof(TO) == 4;
    constexpr int kStep = 2 * kChunk;
    auto acc_wait = [&](int buf, uint32_t n) {
      const bool ok = wait<kTmem>(&s->tfull[buf], (n / kAccs) & 1, abort_flag);
      const bool all = __all_sync(0xffffffffu, ok);
      tc_after();
      return all;
    };
    auto acc_done = [&](int buf) {
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(mapa(smem_u32(&s->tempty[buf]), 0));
    };
    // `take(c, v)` for every 16 of this warp's tokens of the tile, from token c on; false: a wait ran out
    auto boxes = [&](auto halves, auto take) {
      constexpr bool HALVES = decltype(halves)::value;
      const int c0 = half * (HALVES ? kTokens / 2 : kChunk), c1 = HALVES ? min(tl.nj, c0 + kTokens / 2) : tl.nj;
      const auto next = [](int c) { return HALVES || c % kChunk == 0 ? c + 16 : c + kStep - 16; };
      const uint32_t d0 = tmem + ((uint32_t)(32 * q) << 16), sum = d0 + kAccs * kTokens;
      const int chunks = kSums ? ((kAcross ? tl.nk : l.nk) + chunk - 1) / chunk : 1;
      const bool some = !kAcross || tl.nk > 0;                 // else the sums are of no rows: zeros
      for (int ch = 0; ch + 1 < chunks; ++ch, ++acc) {         // all but the last chunk: into the sum's columns
        const int buf = acc % kAccs;
        if (!acc_wait(buf, acc)) return false;
        for (int c = c0; c < c1; c = next(c)) {
          float v[16];
          tmem_ld16(d0 + buf * kTokens + c, v);
          if (ch > 0) {
            float o[16];
            tmem_ld16(sum + c, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += o[j];
          }
          tmem_st16(sum + c, v);
        }
        acc_done(buf);
      }
      const int buf = acc % kAccs;
      if (some) {
        if (!acc_wait(buf, acc)) return false;
        ++acc;
      }
      for (int c = c0; c < c1; c += HALVES ? 2 * 16 : kStep) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[16] = {};
          if (some) tmem_ld16(d0 + buf * kTokens + c + 16 * h, v);
          if (kSums && chunks > 1) {
            float o[16];
            tmem_ld16(sum + c + 16 * h, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += o[j];
          }
          take(c + 16 * h, v);
        }
      }
      if (some) acc_done(buf);
      return true;
    };
    for (int tiles = 1; next_tile(); ++tiles) {
      if (threadIdx.x == 128) *reinterpret_cast<volatile int*>(&s->finishing) = tiles;
      const int f = tl.fti * 2 * kBM + rank * kBM + 32 * q;
      const auto first_row = (kAcross ? (long long)tl.g * l.T : 0) + tl.row0;
      bool ok;
      if (kAcross && p.boxed) {
        // A warp's sums leave by TMA in one box, which leaves out what lies outside, and adds in fp32 where that is asked for.  (Through
        // registers, as below, a tile of 256 x 128 in fp32 took 3.5 us.)
        // In bf16 what is added to comes first, for the sum is rounded once.
        TO* box = reinterpret_cast<TO*>(turn);
        constexpr int kBoxBytes = kBoxTokens<TO> * 32 * (int)sizeof(TO);
        const int c0 = half * (kTokens / 2);
        const bool here = f < l.N && c0 < tl.nj, add = sizeof(TO) == 2 && l.res && here;
        if (lane == 0) store_wait_read<0>();         // the tile before
        if (lane == 0 && add) {
          mbar_expect(&s->old[warp - 4], kBoxBytes);
          tma_3d<1>(smem_u32(box), &p.y, smem_u32(&s->old[warp - 4]), f, tl.row0 + c0, tl.g);
        }
        __syncwarp();
        const auto put = [&](int c, const float (&v)[16]) {
#pragma unroll
          for (int j = 0; j < 16; ++j) box[(c - c0 + j) * 32 + lane] = from_f<TO>(v[j]);
        };
        if (add) {
          bool first = true;
          ok = boxes(std::true_type{}, [&](int c, float (&v)[16]) {
            if (first) wait(&s->old[warp - 4], olds++ & 1, abort_flag);
            first = false;
            float o[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = to_f(box[(c - c0 + j) * 32 + lane]);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += o[j];
            put(c, v);
          });
        } else {
          ok = boxes(std::true_type{}, put);
        }
        fence_async();
        __syncwarp();
        if (lane == 0 && ok && here) {
          if (sizeof(TO) == 4 && l.res)
            tma_store_3d<true>(&p.y, smem_u32(box), f, tl.row0 + c0, tl.g);
          else
            tma_store_3d<false>(&p.y, smem_u32(box), f, tl.row0 + c0, tl.g);
          store_commit();
        }
      } else {
        ok = pair_finish<TO, E4M3>(l, tl.g, first_row, f, tl.nj, half, turn, [&](auto body) {
          return boxes(std::false_type{}, [&](int c, const float (&v)[16]) {
            const int h = c / 16 % 2;
#pragma unroll
            for (int j = 0; j < 16; ++j) turn[(16 * h + j) * 32 + (lane ^ ((j & 7) << 2))] = v[j];
            if (h == 0) return;
            __syncwarp();
            body(c - 16 - half * kChunk);
            __syncwarp();
          });
        });
      }
      if (!ok) break;
    }
    if (kAcross && lane == 0) store_wait_all();
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  settle(abort_flag);
  cluster_sync();                                    // neither CTA's shared memory goes while the other may use it
  tc_after();
  if (warp == 2) tmem_dealloc<2>(tmem, kCols);
  if (kAcross && l.beside) ops_end_beside();
}

// ------------------------------------------------------------------ few tokens

constexpr int kFewTokens = 16;
constexpr int kFewThreads = 512;                     // at most

struct FewParams {
  const void* x;
  const void* w;
  int64_t ldx, ldw;
  LinearParams l;
};

// c[16][8] += a b over 32 bytes of K, twice.  The 16 bytes that a lane loaded of each row (a, and a8 for the
// rows 8 .. of the 16) stand for the same elements in both operands, and no order of K matters to the sum.
template <bool E4M3>
__device__ __forceinline__ void warp_mma(float (&c)[4], const uint4& a, const uint4& a8, const uint4& b) {
#define MOE_WARP_MMA(SHAPE, A0, A1, A2, A3, B0, B1)                                                           \
  asm("mma.sync.aligned." SHAPE " {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"                      \
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                                                        \
      : "r"(A0), "r"(A1), "r"(A2), "r"(A3), "r"(B0), "r"(B1))
  if constexpr (E4M3) {
    MOE_WARP_MMA("m16n8k32.row.col.f32.e4m3.e4m3.f32", a.x, a8.x, a.y, a8.y, b.x, b.y);
    MOE_WARP_MMA("m16n8k32.row.col.f32.e4m3.e4m3.f32", a.z, a8.z, a.w, a8.w, b.z, b.w);
  } else {
    MOE_WARP_MMA("m16n8k16.row.col.f32.bf16.bf16.f32", a.x, a8.x, a.y, a8.y, b.x, b.y);
    MOE_WARP_MMA("m16n8k16.row.col.f32.bf16.bf16.f32", a.z, a8.z, a.w, a8.w, b.z, b.w);
  }
#undef MOE_WARP_MMA
}

// ------------------------------------------------------------------ host side

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// [groups][rows][width] elements of `size` bytes, boxes of 128 bytes x box_rows, 128-byte swizzle,
// zeros outside.
bool encode(CUtensorMap* m, const void* base, int size, int width, int rows, int64_t ld, int groups, int box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)groups};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * size, (cuuint64_t)ld * size * rows};
  const cuuint32_t box[3] = {(cuuint32_t)(kBKBytes / size), (cuuint32_t)box_rows, 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(m, size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, groups > 0 ? 3 : 2,
            const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The windows of 64 rows of a [rows][width] bf16 matrix of 64 rows at least, boxes of 128 bytes x 64 rows, 128-byte swizzle, zeros
// outside the window: element (c, a, b) is column c of row a + b.  All windows lie in the matrix.
bool encode_windows(CUtensorMap* m, const void* base, int width, int rows, int64_t ld) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, kBoxRows, (cuuint64_t)(rows - kBoxRows + 1)}, strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {kBKBytes / 2, kBoxRows, 1}, step[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [groups][rows][width] results, boxes of kBoxTokens rows x 32 elements without swizzle.
template <typename TO>
bool encode_result(CUtensorMap* m, void* base, int width, int rows, int64_t ld, int groups) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)groups};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * sizeof(TO), (cuuint64_t)ld * sizeof(TO) * rows};
  const cuuint32_t box[3] = {32, kBoxTokens<TO>, 1}, step[3] = {1, 1, 1};
  return fn(m, sizeof(TO) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

// k-blocks in the ring of a split CTA that has an SM to itself, or shares one
constexpr int split_stages(int bn, bool own_sm) {
  const int n = ((own_sm ? kSplitSmem : kSplitSmem / 2) - (int)sizeof(SplitTail) - 1024) / (kABlock + bn * kBKBytes);
  return n < SplitTail::kMaxStages ? n : SplitTail::kMaxStages;
}
// the ring holds the CTA's partials and its share of up to 8 ranks' (which may round up by a token each)
constexpr bool split_fits(int bn, bool own_sm) {
  return (bn + bn + 8) * kBM * 4 <= split_stages(bn, own_sm) * (kABlock + bn * kBKBytes);
}
static_assert(split_fits(16, false) && split_fits(32, false) && split_fits(64, false) && split_fits(128, true), "shared memory of the split kernel");

// CTAs of a split kernel, in clusters of s, that find an SM of their own: a cluster stays within its part of the
// chip.  As many again share an SM with another.  `known`: the answers so far, by device.
using Capacities = std::atomic<int>[64][9];
template <class Kernel>
int capacity_of(Kernel kernel, Capacities& known, int s, int sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return sms;
  int n = known[dev][s].load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSplitSmem / 2;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = s;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  // the limit of the launches: another thread may be launching this kernel
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1)
    return sms;
  known[dev][s].store(n * s, std::memory_order_relaxed);
  return n * s;
}
template <int MODE>
int split_capacity(int s, int sms) {
  static Capacities known;
  return capacity_of(linear_split_kernel<false, __nv_bfloat16, MODE>, known, s, sms);      // all forms share its limits
}

struct LinearPlan {
  bool pair;
  int tokens, splits;               // of a tile; CTAs that share its K
};

// Kernel, tile and split with the least expected time, in ns.  The constants are fits to this GPU's timings (some
// 340 shapes and epilogues of 17 to 8192 tokens on 128 to 7168 features, dense and in 8 to 64 groups; the choice's time is
// 1.5% above the best one's on average, 28% at worst).  A k-block costs a split CTA 135 to 230 alone on its SM, by tokens and
// type, and 220 or 280 beside another; a pair 185 to 300.  The exchange takes 100 to 1,300 + 100 a rank, a second CTA on an
// SM 1,100 to 1,900, 128 tokens of a split CTA 2,100 to 3,100, the pair's epilogue 14 a token (30 to 85 element by element)
// behind the last tile, a third more between two.  Neither the epilogue's operands nor strides count: x and w give the same
// sums whatever is done with them.  `bytes`: all operands; the split kernel streams them at 6.4 TB/s, the pair kernel at
// 5.5; of the smaller of stream and sums, part shows.  Groups count half a tile each for their ends.
template <bool E4M3, typename TO, int MODE = kForward>
LinearPlan linear_plan(const LinearParams& l, int sms, float bytes) {
  const float groups = l.offsets ? std::min(l.G, l.T) : 1, per = l.T / groups;
  auto token_tiles = [&](int t) { return l.offsets ? l.T / (float)t + 0.5f * groups : (float)((l.T + t - 1) / t); };
  const int least = per <= 16 ? 16 : per <= 32 ? 32 : 64;
  LinearPlan plan{false, least, 1};
  const bool rows16 = l.N % 8 == 0;
  const float wave = rows16 ? 6600.f : 8300.f;       // a further wave, at least
  float best = 1e30f;
  for (int bn = least; bn == least || (bn == 128 && per > 64); bn *= 2) {
    const float tiles = (l.N + kBM - 1) / kBM * token_tiles(bn);
    for (int s = 1; s <= 8 && (s == 1 || 2 * s <= l.nk); ++s) {
      const float ctas = tiles * s, own = (float)split_capacity<MODE>(s, sms), waves = std::ceil(ctas / (2 * own));
      const bool alone = ctas <= own;
      if ((s > 1 && waves > 1.f) || (bn == 128 && !alone) || (sizeof(TO) == 4 && l.nk > 4 * kChunkBlocks * s)) continue;
      const float kb = (l.nk + s - 1) / s * (!alone ? bn == 64 ? 280.f : 220.f : E4M3 ? bn == 128 ? 230.f : 180.f : bn == 128 ? 157.f : bn == 64 ? 148.f : 135.f);
      const float ns = (s > 1 ? (bn <= 32 ? 3700.f : 4900.f) + 100.f * s : 3600.f) + (bn == 128 ? s > 1 ? 2100.f : 3100.f : 0.f) + (alone ? 0.f : s > 1 ? 1900.f : 1100.f) +
                       (rows16 ? 0.f : 1700.f / s) + kb + (waves - 1) * std::max(kb + 2000.f, wave);
      if (ns < best) best = ns, plan.tokens = bn, plan.splits = s;
    }
  }
  best = std::max(best, 4000.f + bytes / 6400.f) + 0.15f * std::min(best, 4000.f + bytes / 6400.f);
  const float last = rows16 ? 13.7f : sizeof(TO) == 2 ? 30.f : E4M3 ? 85.f : 38.f;      // a token's epilogue
  for (int t = 64; t <= kPairTokens<TO>; t += l.offsets ? t : 32) {
    const float tiles = (l.N + 2 * kBM - 1) / (2 * kBM) * token_tiles(t), rounds = tiles / (sms / 2);
    const float kb = l.nk * std::max(185.f, 90.f + 0.83f * t), finish = 1000.f + 1.3f * last * t;
    float ns = 3600.f + last * t + kb + std::max(0.f, (l.offsets ? rounds : std::ceil(rounds)) - 1.f) * std::max(kb, finish);
    ns = std::max(ns, 5500.f + bytes / 5500.f) + 0.05f * ns;
    if (ns < best) best = ns, plan = {true, t, 1};
  }
  return plan;
}

}  // namespace
}  // namespace moe
