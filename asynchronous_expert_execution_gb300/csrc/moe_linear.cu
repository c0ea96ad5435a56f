// Matrix product with its epilogue, dense or per expert on sorted rows:
//
//   y[t, n] = act(sx[t] sw[n] sum_k x[t, k] w[n, k] + bias[n]) * mul[t, n] + residual[t, n]
//
// x [T, F] and w [N, F] (or [G, N, F]: rows offsets[g] .. offsets[g + 1] of x meet w[g]) in bf16 or
// e4m3, products summed in fp32, y in bf16 or fp32, rounded once.
//
// Weights are the MMA's 128 (or, over two SMs, 256) rows and tokens its columns, so few tokens and
// thousands run on the same tiles: D[feature, token], both operands K-major as they lie in
// memory, tiles of 128 bytes of K by TMA, accumulators in TMEM.  The epilogue passes through
// shared memory as [token][feature]: a thread of a TMEM lane writes its feature's column there,
// and reads back 8 adjacent features of one token, so rows move in 16-byte units (storing from
// the lanes directly, 2 bytes a thread, cost 67,000 cycles a 128 x 256 tile, twice the products
// of a 7168-deep e4m3 tile; turning a whole tile's features at once, with two barriers of 128
// threads per 16 tokens, 17,000).
//
// Three kernels, chosen by expected time (linear_launch, linear_plan):
//   pair   persistent, tiles of 256 features x up to 256 tokens (128 for fp32 results) over two SMs
//          (cta_group::2): each SM stages half of both operands, which halves the shared-memory traffic per product.
//   split  one tile of 128 features x up to 128 tokens per cluster of up to 8 CTAs, K split over
//          them; partials meet through distributed shared memory in rank order (no workspace,
//          no atomics).  For few tiles: a lone SM streams weights far below the HBM rate.
//   few    up to 16 tokens: weights straight into the registers of warp-wide matrix instructions.  Only
//          the weights' bytes count there; barriers, TMEM and the exchange cost more than they bring
//          (4 tokens on 2880 x 2880: 5.8 us against 7.0).
//
// Every wait is bounded (2 s): a wait that runs out stops all roles, latches MOE_ERR_TIMEOUT in
// the operators' error word, and the CTA still lets what is in flight land and frees its TMEM.
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
  __host__ __device__ bool plain() const { return !mul && !res && act == MOE_ACT_NONE; }
};

// Bounded wait; false once it ran out or another role gave up.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try(bar, parity)) return true;
  const unsigned long long t0 = now_ns();
  while (true) {
    if (mbar_try(bar, parity)) return true;
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
__device__ __forceinline__ Span group_rows(const LinearParams& p, int g) {
  if (!p.offsets) return {0, p.T};
  const int a = min(p.T, max(0, __ldg(p.offsets + g))), b = min(p.T, max(a, __ldg(p.offsets + g + 1)));
  return {a, b - a};
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
      for (int u = 0; u < kAt; ++u) got[u] = at + 32 * u + lane < p.G ? group_rows(p, at + 32 * u + lane) : Span{0, 0};
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
template <typename TO>
__device__ __forceinline__ float gelu(float x) {
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
  const float tail = e * (p * t);
  return x * (x < 0.f ? tail : 1.0f - tail);
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
  int bn, stages, splits, nft;      // tokens a tile, ring depth, CTAs a cluster, feature tiles
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
__device__ __forceinline__ void split_finish(const SplitParams& p, int g, int row0, int f0, const float* own, const float* got,
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

template <bool E4M3, typename TO>
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
  if (!l.offsets) {                                  // dense: the tile is known before the inputs are
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
  const int kb0 = (int)((long long)l.nk * rank / p.splits), kb1 = (int)((long long)l.nk * (rank + 1) / p.splits);
  constexpr int kElems = E4M3 ? kBKBytes : kBKBytes / 2;
  const int chunks = min(kAccs, (kb1 - kb0 + kChunkBlocks - 1) / kChunkBlocks);

  if (nj > 0 && warp == 0 && elect()) {
    uint32_t st = 0, phase = 1;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!wait(&s->empty[st], phase, abort_flag)) break;
      const uint32_t a = smem_u32(smem + st * stage_bytes);
      mbar_expect(&s->full[st], stage_bytes);
      tma_3d<1>(a, &p.w, smem_u32(&s->full[st]), kb * kElems, fti * kBM, g);
      tma_2d<1>(a + kABlock, &p.x, smem_u32(&s->full[st]), kb * kElems, row0);
      if (++st == p.stages) st = 0, phase ^= 1;
    }
  } else if (nj > 0 && warp == 1 && elect()) {
    const uint32_t idesc = mma_desc<E4M3>(kBM, p.bn);
    bool ok = true;
    uint32_t st = 0, phase = 0;
    for (int chunk = 0; chunk < chunks && ok; ++chunk) {
      const int n = (kb1 - kb0) * (chunk + 1) / chunks - (kb1 - kb0) * chunk / chunks;
      for (int i = 0; i < n; ++i) {
        if (!(ok = wait(&s->full[st], phase, abort_flag))) break;
        tc_after();
        const uint64_t a = operand_desc(smem_u32(smem + st * stage_bytes));
        mma_block<1, E4M3>(tmem + chunk * p.bn, a, a + (kABlock >> 4), idesc, i > 0);
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
        float v[16];
        tmem_ld16(t + c, v);
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
    if (nj > 0) wait(&s->got, 0, abort_flag);
  } else {
    __syncthreads();
  }
  if (nj > 0) {                                      // every rank sums and finishes its share of the tokens
    if (l.wide)
      split_finish<TO, 8, E4M3>(p, g, row0, fti * kBM, own, got, rank, j0, j1, threadIdx.x % 16 * 8, 1, threadIdx.x / 16, kThreads / 16);
    else
      split_finish<TO, 4, E4M3>(p, g, row0, fti * kBM, own, got, rank, j0, j1, lane, 32, warp, kThreads / 32);
  }
  settle(abort_flag);
  if (p.splits > 1) cluster_sync();                  // the copies out of a rank's memory have been received
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 2) tmem_dealloc<1>(tmem, cols);
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

struct PairParams {
  CUtensorMap w, x[4];              // x: boxes of 16, 32, 64 and tokens / 2 rows
  LinearParams l;
  int nft;                          // feature tiles of 256
  int tokens;                       // of a tile, a multiple of 32
  int stages, stage_bytes;          // of the ring: a k-block of a full tile each
};

struct PairTail {
  static constexpr int kMaxStages = 10;
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[4], tempty[4];
  uint32_t tmem;
  int abort_flag;
  int finishing;                    // tiles whose epilogue has begun
};

struct PairTile {
  int g, row0, nj, fti, nmma, box, brows;   // brows: token rows a CTA stages
};

// The tiles of a pair of CTAs, in order: every `pairs`-th one.  Every role's warp walks the groups by itself.  Groups
// with a full tile come first, then those with more than half of one: long tiles at the end would leave pairs idle
// (2880 x 2880, 32 groups of 18 to 1151 rows: 138 us, in the groups' order 142; e4m3 88 and 92; 64 groups of 2048 x
// 768 on 16384 rows 66 and 73).
struct PairWalk {
  GroupTiles at;
  int pass = 0;
  __device__ __forceinline__ PairWalk() : at(blockIdx.x / 2) {}

  // by whole warps
  __device__ __forceinline__ bool next(const PairParams& p, PairTile& tl) {
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

template <bool E4M3, typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ PairParams p) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  PairTail* s = reinterpret_cast<PairTail*>(smem + kPairRing + kStaging);
  volatile int* abort_flag = &s->abort_flag;
  const LinearParams& l = p.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  constexpr int kTokens = kPairTokens<TO>, kAccs = sizeof(TO) == 4 ? 3 : 2;
  constexpr uint32_t kCols = 512;
  const int chunk = sizeof(TO) == 4 ? kChunkBlocks : l.nk;      // k-blocks summed in one accumulator

  if (threadIdx.x == 0) {
    prefetch_map(&p.w);
    prefetch_map(&p.x[3]);
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&s->full[i], 1);                     // the leader's producer, for both CTAs' bytes
      mbar_init(&s->empty[i], 1);                    // the MMA's commit, in both CTAs
    }
    for (int b = 0; b < kAccs; ++b) {
      mbar_init(&s->tfull[b], 1);
      mbar_init(&s->tempty[b], 16);                  // the epilogue warps of both CTAs, at the leader
    }
    s->abort_flag = 0;
    s->finishing = 0;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc<2>(&s->tmem, kCols);
  ops_begin();
  tc_before();
  __syncthreads();
  cluster_sync();
  tc_after();
  const uint32_t tmem = s->tmem;
  PairWalk walk;
  PairTile tl;
  constexpr int kElems = E4M3 ? kBKBytes : kBKBytes / 2;

  if (warp == 0) {
    uint32_t st = 0, phase = 1;
    bool ok = true;
    while (__all_sync(0xffffffffu, ok) && walk.next(p, tl)) {
      if (!elect()) continue;
      const int block = kABlock + tl.brows * kBKBytes;
      const int wrow = tl.fti * 2 * kBM + rank * kBM, xrow = tl.row0 + rank * (tl.nmma / 2);
      for (int kb = 0; kb < l.nk; ++kb) {
        if (!(ok = wait(&s->empty[st], phase, abort_flag))) break;
        const uint32_t a = smem_u32(smem + st * p.stage_bytes), bar = mapa(smem_u32(&s->full[st]), 0);
        if (rank == 0) mbar_expect(&s->full[st], 2 * block);
        tma_3d<2>(a, &p.w, bar, kb * kElems, wrow, tl.g);
        tma_2d<2>(a + kABlock, &p.x[tl.box], bar, kb * kElems, xrow);
        if (++st == p.stages) st = 0, phase ^= 1;
      }
    }
  } else if (warp == 1 && rank == 0) {
    uint32_t st = 0, phase = 0, acc = 0;
    bool ok = true;
    while (__all_sync(0xffffffffu, ok) && walk.next(p, tl)) {
      if (!elect()) continue;
      const uint32_t idesc = mma_desc<E4M3>(2 * kBM, tl.nmma);
      int buf = 0;
      for (int kb = 0, in = chunk; kb < l.nk; ++kb, ++in) {      // in: k-blocks in this accumulator
        if (in == chunk) {
          if (kb > 0) commit<2>(&s->tfull[buf]);
          buf = acc % kAccs;
          if (!(ok = wait(&s->tempty[buf], ((acc / kAccs) & 1) ^ 1, abort_flag))) break;
          tc_after();
          ++acc;
          in = 0;
        }
        if (!(ok = wait(&s->full[st], phase, abort_flag))) break;
        tc_after();
        const uint64_t a = operand_desc(smem_u32(smem + st * p.stage_bytes));
        mma_block<2, E4M3>(tmem + buf * kTokens, a, a + (kABlock >> 4), idesc, in > 0);
        commit<2>(&s->empty[st]);
        if (++st == p.stages) st = 0, phase ^= 1;
      }
      if (ok) commit<2>(&s->tfull[buf]);
    }
  } else if (warp == 3 && (l.mul || l.res)) {
    // mul and residual of a tile into L2 while the tile before is finished: the epilogue's 16 KB of
    // reads in flight an SM then last L2's latency (4096 x 512 x 7168 with mul: 50 -> 45 us)
    volatile int* finishing = &s->finishing;
    for (int i = 0; walk.next(p, tl); ++i) {
      const unsigned long long t0 = now_ns();
      while (*finishing < i && !*abort_flag && now_ns() - t0 < kLimitNs) __nanosleep(200);
      const int f = tl.fti * 2 * kBM + rank * kBM, n = min(kBM, l.N - f) * (int)sizeof(TO), lines = kBM * (int)sizeof(TO) / 128;
      for (int j = lane / lines; j < tl.nj; j += 32 / lines) {
        const int64_t r = tl.row0 + j;
        if (lane % lines * 128 < n) {
          if (l.mul) prefetch_l2(reinterpret_cast<const char*>(static_cast<const TO*>(l.mul) + r * l.ldmul + f) + lane % lines * 128);
          if (l.res) prefetch_l2(reinterpret_cast<const char*>(static_cast<const TO*>(l.res) + r * l.ldres + f) + lane % lines * 128);
        }
      }
    }
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp >> 2) - 1;  // TMEM lanes 32 q ..; two warps share a quarter's columns
    float* turn = reinterpret_cast<float*>(smem + kPairRing) + (warp - 4) * kTurn;
    uint32_t acc = 0;
    // a warp's tokens: every other block of 32
    constexpr bool kSums = sizeof(TO) == 4;
    constexpr int kStep = 2 * kChunk;
    auto acc_wait = [&](int buf, uint32_t n) {
      const bool ok = wait(&s->tfull[buf], (n / kAccs) & 1, abort_flag);
      const bool all = __all_sync(0xffffffffu, ok);
      tc_after();
      return all;
    };
    auto acc_done = [&](int buf) {
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa(smem_u32(&s->tempty[buf]), 0));
    };
    // `body(c)` for each of this warp's blocks of the tile, the block's sums in `turn`; false: a wait ran out
    auto blocks = [&](auto body) {
      const uint32_t d0 = tmem + ((uint32_t)(32 * q) << 16), sum = d0 + kAccs * kTokens;
      const int chunks = kSums ? (l.nk + chunk - 1) / chunk : 1;
      for (int ch = 0; ch + 1 < chunks; ++ch, ++acc) {         // all but the last chunk: into the sum's columns
        const int buf = acc % kAccs;
        if (!acc_wait(buf, acc)) return false;
        for (int c = half * kChunk; c < tl.nj; c += c % kChunk ? kStep - 16 : 16) {
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
      if (!acc_wait(buf, acc)) return false;
      ++acc;
      for (int c = half * kChunk; c < tl.nj; c += kStep) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[16];
          tmem_ld16(d0 + buf * kTokens + c + 16 * h, v);
          if (kSums && chunks > 1) {
            float o[16];
            tmem_ld16(sum + c + 16 * h, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += o[j];
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) turn[(16 * h + j) * 32 + (lane ^ ((j & 7) << 2))] = v[j];
        }
        __syncwarp();
        body(c - half * kChunk);
        __syncwarp();
      }
      acc_done(buf);
      return true;
    };
    for (int tiles = 1; walk.next(p, tl); ++tiles) {
      if (threadIdx.x == 128) *reinterpret_cast<volatile int*>(&s->finishing) = tiles;
      const int f = tl.fti * 2 * kBM + rank * kBM + 32 * q;
      bool ok;
      const auto wide = [&](auto plain) {
        constexpr bool PLAIN = decltype(plain)::value;
        // 32 features x 32 tokens turned in the warp's own shared memory: lane i then holds 8
        // features (i % 4) of tokens i / 4 + 8 u, u < 4.  16-byte chunks of a token's row lie at
        // chunk ^ (token & 7): neither the writes nor the reads meet a bank twice.  mul and
        // residual are asked for kAt units ahead, the first ones before the products are done.
        constexpr int kAt = kSums ? 2 : 4, kU = PLAIN ? 2 : 1;         // kU units at once: more would delay the next loads
        const int f8 = lane % 4, tk = lane / 4;
        const Finish<TO, 8, E4M3, PLAIN> finish(l, tl.g, f + f8 * 8, 1);
        const Place<TO> place(l, tl.row0 + half * kChunk + tk, f + f8 * 8);
        const int mine = tl.nj - half * kChunk - tk;           // tokens from this lane's first to the tile's end
        typename Finish<TO, 8, E4M3, PLAIN>::Ahead a[kAt];
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
        ok = l.plain() ? wide(std::true_type{}) : wide(std::false_type{});
      } else {
        // a lane keeps its feature: 32 adjacent elements of a token a warp, kAt tokens at once
        const auto narrow = [&](auto plain) {
          constexpr bool PLAIN = decltype(plain)::value;
          constexpr int kAt = kSums ? PLAIN || E4M3 ? 2 : 8 : PLAIN || E4M3 ? 8 : 16;
          using F = Finish<TO, 1, E4M3, PLAIN>;
          const F finish(l, tl.g, f + lane, 1);
          const Place<TO> place(l, tl.row0 + half * kChunk, f + lane);
          const int mine = tl.nj - half * kChunk;
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
        ok = l.plain() ? narrow(std::true_type{}) : narrow(std::false_type{});
      }
      if (!ok) break;
    }
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  settle(abort_flag);
  cluster_sync();                                    // neither CTA's shared memory goes while the other may use it
  tc_after();
  if (warp == 2) tmem_dealloc<2>(tmem, kCols);
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

// An SM's share of HBM, 45 GB/s, wants some 40 KB under way: 512 threads ask for eight (FS + TS = 2), five or four
// 16-byte units a row each before they use the first.  Sums on the CUDA cores instead took 6.5 us for one
// token on 2880 x 2880 (5.8 here) and 17.6 for eight (6.0).
// Block (b, i): 8 FS features of up to 8 TS tokens, those of the i-th group that has rows.  Each of its W
// warps takes every W-th 64 bytes of K, kAhead of them in flight; their sums meet in shared memory and
// are added in order.
template <bool E4M3, typename TO, int TS, int FS>
__global__ void __launch_bounds__(kFewThreads, 1) linear_few_kernel(const __grid_constant__ FewParams p) {
  constexpr int kSize = E4M3 ? 1 : 2, kAhead = 16 / (TS + FS), kFeatures = 8 * FS;
  __shared__ float part[kFewThreads / 32][8 * TS * kFeatures];
  ops_begin();
  const LinearParams& l = p.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  int g = 0, row0 = 0, nt = l.T;
  if (l.offsets) {
    nt = 0;
    const auto tiles = [](int n) { return n > 0 ? 1 : 0; };
    GroupTiles at(blockIdx.y);
    if (at.find(l, tiles)) at.get(tiles, g, row0, nt);
    nt = min(8 * TS, nt);
    if (nt == 0) return;
  }
  // this thread's output, and what its epilogue reads
  const int of = blockIdx.x * kFeatures + threadIdx.x % kFeatures, ot = threadIdx.x / kFeatures;
  const bool out = ot < nt;
  const Finish<TO, 1, E4M3> finish(l, g, out ? of : l.N, 1);
  const Place<TO> place(l, row0 + ot, of);
  typename Finish<TO, 1, E4M3>::Ahead ahead;
  finish.ahead(ahead, place, 0, out);

  // rows in units of 16 bytes; a row that does not exist is not read
  const int units = (int)((int64_t)l.F * kSize / 16);
  const uint4 *w[FS], *x[TS];
  int wu[FS], xu[TS];
#pragma unroll
  for (int i = 0; i < FS; ++i) {
    const int f = blockIdx.x * kFeatures + i * 8 + lane / 4;
    wu[i] = f < l.N ? units : 0;
    w[i] = static_cast<const uint4*>(p.w) + ((size_t)g * l.N + (f < l.N ? f : 0)) * (p.ldw * kSize / 16);
  }
#pragma unroll
  for (int i = 0; i < TS; ++i) {
    const int t = i * 8 + lane / 4;
    xu[i] = t < nt ? units : 0;
    x[i] = static_cast<const uint4*>(p.x) + (row0 + (t < nt ? t : 0)) * (size_t)(p.ldx * kSize / 16);
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  constexpr int kTiles = TS * FS == 4 ? 2 : 1;       // of 16 x 8 sums
  float sum[kTiles][4] = {};
  for (int k0 = warp * 4; k0 < units; k0 += kAhead * warps * 4) {
    uint4 wv[FS][kAhead], xv[TS][kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = k0 + lane % 4 + u * warps * 4;
#pragma unroll
      for (int i = 0; i < FS; ++i) wv[i][u] = k < wu[i] ? __ldcs(w[i] + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = k0 + lane % 4 + u * warps * 4;
#pragma unroll
      for (int i = 0; i < TS; ++i) xv[i][u] = k < xu[i] ? __ldg(x[i] + k) : zero;
    }
    // the matrix instruction truncates as it adds: short sums there, their sum here
    float c[kTiles][4] = {};
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if constexpr (FS == 2) {
#pragma unroll
        for (int i = 0; i < TS; ++i) warp_mma<E4M3>(c[i], wv[0][u], wv[1][u], xv[i][u]);
      } else {
        warp_mma<E4M3>(c[0], xv[0][u], TS == 2 ? xv[TS - 1][u] : zero, wv[0][u]);
      }
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[i][j] += c[i][j];
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = lane / 4 + j / 2 * 8, q = i * 8 + lane % 4 * 2 + j % 2;
      if (FS == 2) part[warp][q * kFeatures + r] = sum[i][j];
      else if (TS == 2 || j < 2) part[warp][r * kFeatures + q] = sum[i][j];
    }
  __syncthreads();
  if (out) {
    float v[1] = {part[0][threadIdx.x]};
    for (int i = 1; i < warps; ++i) v[0] += part[i][threadIdx.x];
    finish(v, place.y, ahead);
  }
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

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

template <bool E4M3, typename TO>
moe_status launch_pair(const moe_async_linear_args* a, const LinearParams& l, int sms, int tokens, void* s) {
  constexpr int kSmem = kPairRing + kStaging + (int)sizeof(PairTail) + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  constexpr int size = E4M3 ? 1 : 2;
  PairParams p;
  p.l = l;
  p.nft = (l.N + 2 * kBM - 1) / (2 * kBM);
  if (!encode(&p.w, a->d_w, size, l.F, l.N, a->w_stride, l.G, kBM)) return MOE_ERR_CUDA;
  p.tokens = tokens;
  p.stage_bytes = kABlock + tokens / 2 * kBKBytes;
  p.stages = std::min(PairTail::kMaxStages, kPairRing / p.stage_bytes);
  for (int i = 0; i < 4; ++i)
    if (!encode(&p.x[i], a->d_x, size, l.F, l.T, a->x_stride, 0, i < 3 ? 16 << i : tokens / 2)) return MOE_ERR_CUDA;
  if (cudaFuncSetAttribute(linear_pair_kernel<E4M3, TO>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
    return MOE_ERR_CUDA;
  return launch_op(linear_pair_kernel<E4M3, TO>, dim3(sms / 2 * 2), kPairThreads, kSmem, 1, s, p);
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

// CTAs of the split kernel, in clusters of s, that find an SM of their own: a cluster stays within its part of the
// chip.  As many again share an SM with another.
int split_capacity(int s, int sms) {
  static std::atomic<int> known[64][9];
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
  const auto kernel = linear_split_kernel<false, __nv_bfloat16>;       // all forms share its limits
  // the limit of launch_split: another thread may be launching this kernel
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1)
    return sms;
  known[dev][s].store(n * s, std::memory_order_relaxed);
  return n * s;
}

template <bool E4M3, typename TO>
moe_status launch_split(const moe_async_linear_args* a, const LinearParams& l, int bn, int splits, int64_t tiles, int sms, void* s) {
  constexpr int size = E4M3 ? 1 : 2;
  SplitParams p;
  p.l = l;
  p.bn = bn;
  p.splits = splits;
  p.nft = (l.N + kBM - 1) / kBM;
  // Alone on its SM a CTA takes all of the shared memory where its K fills it, for loads in flight (512 x 7168 x 256: 10.7 ->
  // 8.9 us); two CTAs on an SM fill each other's gaps.  128 tokens' accumulators and partials fit one CTA an SM only.
  p.stages = split_stages(bn, false);
  if (bn > 64 || (tiles * splits <= split_capacity(splits, sms) && l.nk > p.stages * splits)) p.stages = split_stages(bn, true);
  const int stage = kABlock + bn * kBKBytes, rest = (int)sizeof(SplitTail) + 1024;
  const int smem = p.stages * stage + rest;
  if (!encode(&p.w, a->d_w, size, l.F, l.N, a->w_stride, l.G, kBM) ||
      !encode(&p.x, a->d_x, size, l.F, l.T, a->x_stride, 0, bn))
    return MOE_ERR_CUDA;
  if (cudaFuncSetAttribute(linear_split_kernel<E4M3, TO>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmem) != cudaSuccess)
    return MOE_ERR_CUDA;
  return launch_op(linear_split_kernel<E4M3, TO>, dim3((unsigned)(tiles * splits)), kThreads, smem, splits, s, p);
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
template <bool E4M3, typename TO>
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
      const float ctas = tiles * s, own = (float)split_capacity(s, sms), waves = std::ceil(ctas / (2 * own));
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

template <bool E4M3, typename TO, int TS, int FS>
moe_status launch_few(const moe_async_linear_args* a, const LinearParams& l, int sms, void* s) {
  const FewParams p{a->d_x, a->d_w, a->x_stride, a->w_stride, l};
  const dim3 grid((unsigned)((l.N + 8 * FS - 1) / (8 * FS)), (unsigned)(l.offsets ? std::min(l.G, l.T) : 1));
  // Twice the warps where a block has an SM to itself and half of them would take K in more than one pass (1 token on
  // 7168 x 256: 4.4 us against 6.4; but on 512 x 256 2.0 against 1.7, on 2880 x 2880 7.9 against 5.8)
  const bool one_pass = (int64_t)l.F * (E4M3 ? 1 : 2) <= kFewThreads / 64 * 64 * (16 / (TS + FS));
  const int threads = one_pass || grid.x * grid.y > (unsigned)sms ? kFewThreads / 2 : kFewThreads;
  return launch_op(linear_few_kernel<E4M3, TO, TS, FS>, grid, threads, 0, 1, s, p);
}

template <bool E4M3, typename TO>
moe_status linear_launch(const moe_async_linear_args* a, const LinearParams& l, void* s) {
  const int sms = sm_count();
  if (sms < 2) return MOE_ERR_CUDA;
  // Up to 16 tokens the few kernel is ahead on small weights (bf16, few / split us: 1 token on 2880 x 2880 5.8 / 6.9, 7168 x
  // 256 4.4 / 6.1, 512 x 256 1.7 / 3.9, 7168 x 4096 12.4 / 13.3; 16 tokens 6.1 / 7.2, 6.2 / 6.4, 1.8 / 3.9, 13.0 / 13.6;
  // e4m3, 8 tokens of 8 of 128 groups on 2048 x 768 5.8 / 7.9), until its blocks are many (1 token on 512 x 30000 11.9 /
  // 8.0) or its re-reads of x crowd a long stream (1 token on 6144 x 6144 17.3 / 15.9, 16 tokens 20.2 / 16.5).
  const int64_t features = (int64_t)l.N * (l.offsets ? std::min(l.G, l.T) : 1);
  if (l.T <= kFewTokens && features <= 64 * sms && features * l.F <= 32'000'000) {
    // 16 features a block re-read x half as often (1 token on 2880 x 2880 5.8 us against 7.2; 16 tokens 6.1 against
    // 9.0), 8 make enough blocks of a small weight (1 token on 7168 x 1024 6.5 against 5.4)
    const bool wide = features > 8 * sms;
    return l.T > 8 ? wide ? launch_few<E4M3, TO, 2, 2>(a, l, sms, s) : launch_few<E4M3, TO, 2, 1>(a, l, sms, s)
                   : wide ? launch_few<E4M3, TO, 1, 2>(a, l, sms, s) : launch_few<E4M3, TO, 1, 1>(a, l, sms, s);
  }
  const LinearPlan plan = linear_plan<E4M3, TO>(l, sms, ((float)features + l.T) * l.F * (E4M3 ? 1 : 2));
  if (plan.pair) return launch_pair<E4M3, TO>(a, l, sms, plan.tokens, s);
  const int64_t tiles = (int64_t)((l.N + kBM - 1) / kBM) * (l.offsets ? l.T / plan.tokens + std::min(l.G, l.T) : (l.T + plan.tokens - 1) / plan.tokens);
  return launch_split<E4M3, TO>(a, l, plan.tokens, plan.splits, tiles, sms, s);
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_async_linear(const moe_async_linear_args* a, void* stream) {
  using namespace moe;
  if (!a) return MOE_ERR_INVALID;
  if (a->rows < 0 || a->rows > INT32_MAX - 1024 || a->fan_in < 1 || a->fan_in > INT32_MAX - 1024 ||
      a->fan_out < 1 || a->fan_out > INT32_MAX - 1024 || a->groups < 0 || a->groups > kMaxExperts ||
      a->act < MOE_ACT_NONE || a->act > MOE_ACT_RELU || (a->groups > 0) != (a->d_offsets != nullptr) ||
      (a->out_dtype != MOE_F32 && a->out_dtype != MOE_BF16))
    return MOE_ERR_INVALID;
  if (a->dtype != MOE_BF16 && a->dtype != MOE_E4M3) return MOE_ERR_UNSUPPORTED;
  if (a->rows == 0) return MOE_OK;
  const int size = dtype_size(a->dtype);
  const bool e4m3 = a->dtype == MOE_E4M3;
  if (!a->d_x || !a->d_w || !a->d_y || a->x_stride < a->fan_in || a->w_stride < a->fan_in || a->y_stride < a->fan_out ||
      (a->d_mul && a->mul_stride < a->fan_out) || (a->d_residual && a->residual_stride < a->fan_out) ||
      (a->d_x_scale != nullptr) != e4m3 || (a->d_w_scale != nullptr) != e4m3)
    return MOE_ERR_INVALID;
  // the operands move in 16-byte units
  if ((int64_t)a->fan_in * size % 16 || !rows16(a->d_x, a->x_stride, size) || !rows16(a->d_w, a->w_stride, size))
    return MOE_ERR_UNSUPPORTED;
  const int os = dtype_size(a->out_dtype);
  const bool wide = a->fan_out % 8 == 0 && rows16(a->d_y, a->y_stride, os) && rows16(a->d_mul, a->mul_stride, os) &&
                    rows16(a->d_residual, a->residual_stride, os);
  const LinearParams l{a->d_bias,   a->d_x_scale,  a->d_w_scale,       a->d_mul,
                       a->d_residual, a->d_y,      a->d_offsets,       a->mul_stride,
                       a->residual_stride, a->y_stride, a->rows,       a->fan_out,
                       a->fan_in,   std::max(1, a->groups), a->act,    (int)(((int64_t)a->fan_in * size + kBKBytes - 1) / kBKBytes), wide};
  if (e4m3)
    return a->out_dtype == MOE_BF16 ? linear_launch<true, __nv_bfloat16>(a, l, stream)
                                    : linear_launch<true, float>(a, l, stream);
  return a->out_dtype == MOE_BF16 ? linear_launch<false, __nv_bfloat16>(a, l, stream)
                                  : linear_launch<false, float>(a, l, stream);
}

extern "C" moe_status moe_async_ops_status(void* stream) {
  using namespace moe;
  unsigned int e = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyFromSymbolAsync(&e, g_ops_error, sizeof(e), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (e == 0) return MOE_OK;
  const unsigned int none = 0;                       // reported: the calls after this one start clear
  if (cudaMemcpyToSymbolAsync(g_ops_error, &none, sizeof(none), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return MOE_ERR_CUDA;
  return static_cast<moe_status>(e);
}

extern "C" moe_status moe_async_debug_latch_ops_error(void* stream) {
#ifdef MOE_DEBUG_BOUNDS
  using namespace moe;
  const unsigned int e = MOE_ERR_TIMEOUT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cudaMemcpyToSymbolAsync(g_ops_error, &e, sizeof(e), 0, cudaMemcpyHostToDevice, s) == cudaSuccess &&
                 cudaStreamSynchronize(s) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
#else
  (void)stream;
  return MOE_ERR_UNSUPPORTED;
#endif
}
