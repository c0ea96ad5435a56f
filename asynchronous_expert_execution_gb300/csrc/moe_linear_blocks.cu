// The product of e4m3 operands with a scale per 128 columns of a token and per 128 x 128 block of a weight, dense or
// per expert on sorted rows, and the quantisers that make such operands:
//
//   v[t, n] = sum_b sx[t, b] sw[n / 128, b] sum_{k in block b} x[t, k] w[n, k],   b = k / 128
//
// then the epilogue of the forward product (moe_linear.cuh): act(v + bias) * mul + residual.
//
// 128 e4m3 columns are one k-block (128 bytes, one swizzle atom), so every k-block's sum stands under one scale a token
// and feature block.  The tensor cores sum a k-block into a TMEM buffer of its own, and the epilogue warps, while the
// next ones are summed, bring it into their registers times sx sw: the sum over blocks is rounded in fp32 (the tensor
// cores' own sums of four instructions are too short for their cut to show).  128 features are one block of w's scales, so
// sx sw is one number a token, which a warp lays into shared memory ahead of use.
//
//   pair   persistent, 256 tokens x 256 features over two SMs, tokens on the MMA's rows; for many tokens
//   split  128 features x up to 64 tokens, features on the MMA's rows as in the forward product, K split over a cluster of up to 8 CTAs
//   few    up to 16 tokens on small weights, by warp-wide matrix instructions
// 4096 x 7168 x 7168 in bf16 takes 201 us with a residual (2.1 PFLOP/s, 56% of twice the measured bf16 rate), 175 without; 256 x 7168 x 2048
// 16, 4 x 7168 x 2048 5.3.
#include "moe_linear.cuh"

namespace moe {
namespace {

// acc[0 .. 16) += 16 columns times their tokens' factors, which lie in shared memory.  (Multiply-adds on pairs, fma.f32x2, run no
// faster, and bringing what was read from TMEM into pairs cost more than they: 128 columns by two warps of a scheduler 1,035 cycles,
// so 356.)
__device__ __forceinline__ void take(float* acc, const float (&d)[16], uint32_t factor) {
#pragma unroll
  for (int j = 0; j < 16; j += 4) {
    float f[4];
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(factor + 4 * j));
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j + i] = fmaf(d[j + i], f[i], acc[j + i]);
  }
}

// Scales of x, [rows][blocks] with any strides, and of w, [groups][feature blocks][blocks].
struct Scales {
  const float* x;
  const float* w;
  int64_t row, block;
  int nfb;
};

constexpr int kBatch = 4;                            // k-blocks whose factors are loaded together

// A warp lays sx sw of `n` tokens from `row` on into shared memory, kBatch k-blocks to a slot, whose loads are in flight together.
template <int SLOTS, int TOKENS, class Ready>
__device__ __forceinline__ void lay_factors(const Scales& sc, const LinearParams& l, int g, int fb, int row, int n, int kb0, int kb1,
                                            float (*slot)[kBatch][TOKENS], uint64_t* full, uint32_t& at, Ready wait_empty) {
  constexpr int kPer = (TOKENS + 31) / 32;
  const int lane = threadIdx.x & 31;
  const float* sw = sc.w + ((size_t)g * sc.nfb + min(fb, sc.nfb - 1)) * l.nk;
  const float* sx = sc.x + (int64_t)(row + lane) * sc.row;
  for (int kb = kb0; kb < kb1; kb += kBatch, ++at) {
    float v[kBatch][kPer];
    const float mine = lane < kBatch && kb + lane < kb1 ? __ldg(sw + kb + lane) : 0.f;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const float* from = sx + (kb + b) * sc.block;
#pragma unroll
      for (int i = 0; i < kPer; ++i, from += 32 * sc.row) v[b][i] = kb + b < kb1 && lane + 32 * i < n ? __ldg(from) : 0.f;
    }
    const int s = at % SLOTS;
    if (!wait_empty(s, ((at / SLOTS) & 1) ^ 1)) return;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const float w = __shfl_sync(0xffffffffu, mine, b);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (TOKENS % 32 == 0 || lane + 32 * i < TOKENS) slot[s][b][lane + 32 * i] = v[b][i] * w;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[s]);
  }
}

// ------------------------------------------------------------------ pair kernel

// Tokens are the MMA's rows here, and so the lanes of TMEM: a thread has one token, and one factor for all of a k-block's 128
// features that it adds.  With features on the lanes, as in the split kernel, every column has a factor of its own, and their reads of
// shared memory (one of 16 bytes for four columns a warp) held a k-block of 256 x 256 to 965 cycles where the products take some 570.
// The price is that a group's last tile is summed as if it were full.
constexpr int kBlockRing = 160 * 1024;
constexpr int kTileSlots = 4, kFactorSlots = 3;
// registers: the launch gives every thread 168; the epilogue's warps, which hold a tile's sums, take from the others
constexpr int kLaunchRegs = 168, kFewRegs = 72, kManyRegs = 216;
static_assert(128 * kFewRegs + 256 * kManyRegs <= kPairThreads * kLaunchRegs, "the warps' registers are those of the launch");

struct BlockPairParams {
  PairParams p;                     // x[3]: boxes of 128 tokens
  Scales s;
};

struct BlockPairTail {
  static constexpr int kStages = kBlockRing / (2 * kABlock);
  float factor[kFactorSlots][kBatch][2][kBM];        // of either half's features and a token
  uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], told[kTileSlots], heard[kTileSlots], sfull[kFactorSlots], sempty[kFactorSlots];
  int4 tile[kTileSlots];            // g, first row, rows, feature tile; no rows: there are no more
  uint32_t tmem;
  int abort_flag;
};
constexpr int kBlockPairSmem = kBlockRing + kStaging + (int)sizeof(BlockPairTail) + 1024;
static_assert(kBlockPairSmem <= 227 * 1024, "shared memory of a CTA");

template <typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_blocks_pair_kernel(const __grid_constant__ BlockPairParams bp) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  using Tail = BlockPairTail;
  Tail* s = reinterpret_cast<Tail*>(smem + kBlockRing + kStaging);
  volatile int* abort_flag = &s->abort_flag;
  const PairParams& p = bp.p;
  const LinearParams& l = p.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  constexpr uint32_t kCols = 512;
  constexpr int kStage = 2 * kABlock;

  if (threadIdx.x == 0) {
    prefetch_map(&p.w);
    prefetch_map(&p.x[3]);
    for (int i = 0; i < Tail::kStages; ++i) {
      mbar_init(&s->full[i], 1);                     // the leader's producer, for both CTAs' bytes
      mbar_init(&s->empty[i], 1);                    // the MMA's commit, in both CTAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s->tfull[b], 1);
      mbar_init(&s->tempty[b], 16);                  // the epilogue warps of both CTAs, at the leader
    }
    for (int i = 0; i < kTileSlots; ++i) {
      mbar_init(&s->told[i], 1);
      mbar_init(&s->heard[i], 8);
    }
    for (int i = 0; i < kFactorSlots; ++i) {
      mbar_init(&s->sfull[i], 1);
      mbar_init(&s->sempty[i], 8);
    }
    s->abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc<2>(&s->tmem, kCols);
  ops_begin();
  tc_before();
  __syncthreads();
  cluster_sync();
  tc_after();
  const uint32_t tmem = s->tmem;

  if (warp < 4) {
    regs_give<kFewRegs>();
    PairWalk walk;
    PairTile tl;
    if (warp == 0) {
      uint32_t st = 0, phase = 1;
      bool ok = true;
      while (__all_sync(0xffffffffu, ok) && walk.next<kForward>(p, tl)) {
        if (!elect()) continue;
        const int wrow = tl.fti * 2 * kBM + rank * kBM, xrow = tl.row0 + rank * kBM;
        for (int kb = 0; kb < l.nk; ++kb) {
          if (!(ok = wait<kCluster>(&s->empty[st], phase, abort_flag))) break;
          const uint32_t a = smem_u32(smem + st * kStage), bar = mapa(smem_u32(&s->full[st]), 0);
          if (rank == 0) mbar_expect(&s->full[st], 2 * kStage);
          tma_2d<2>(a, &p.x[3], bar, kb * kBKBytes, xrow);
          tma_3d<2>(a + kABlock, &p.w, bar, kb * kBKBytes, wrow, tl.g);
          if (++st == Tail::kStages) st = 0, phase ^= 1;
        }
      }
    } else if (warp == 1 && rank == 0) {
      uint32_t st = 0, phase = 0, acc = 0;
      bool ok = true;
      const uint32_t idesc = mma_desc<true>(2 * kBM, 2 * kBM);
      while (__all_sync(0xffffffffu, ok) && walk.next<kForward>(p, tl)) {
        if (!elect()) continue;
        for (int kb = 0; kb < l.nk; ++kb, ++acc) {
          if (!(ok = wait<kCluster>(&s->full[st], phase, abort_flag))) break;
          const uint64_t a = operand_desc(smem_u32(smem + st * kStage));
          const int buf = acc & 1;
          if (!(ok = wait<kTmem>(&s->tempty[buf], ((acc >> 1) & 1) ^ 1, abort_flag))) break;
          tc_after();
          mma_block<2, true>(tmem + buf * 2 * kBM, a, a + (kABlock >> 4), idesc, false);
          commit<2>(&s->empty[st]);
          commit<2>(&s->tfull[buf]);
          if (++st == Tail::kStages) st = 0, phase ^= 1;
        }
      }
    } else if (warp == 2) {
      // tells the epilogue its tiles, whose registers have no room for the walk, and pulls a tile's mul and residual into L2 while it is
      // summed: the epilogue's reads in flight an SM then last L2's latency
      for (uint32_t n = 0, more = 1; more; ++n) {
        const int slot = n % kTileSlots;
        more = walk.next<kForward>(p, tl);
        if (!__all_sync(0xffffffffu, wait(&s->heard[slot], ((n / kTileSlots) & 1) ^ 1, abort_flag))) break;
        if (lane == 0) {
          s->tile[slot] = make_int4(tl.g, tl.row0, more ? tl.nj : 0, tl.fti);
          mbar_arrive(&s->told[slot]);
        }
        __syncwarp();
        if (more && (l.mul || l.res)) {
          const int f = tl.fti * 2 * kBM, width = min(2 * kBM, l.N - f) * (int)sizeof(TO), lines = 2 * kBM * (int)sizeof(TO) / 128;
          for (int j = rank * kBM + lane / lines; j < min(tl.nj, (rank + 1) * kBM); j += 32 / lines) {
            const int64_t r = tl.row0 + j;
            if (lane % lines * 128 < width) {
              if (l.mul) prefetch_l2(reinterpret_cast<const char*>(static_cast<const TO*>(l.mul) + r * l.ldmul + f) + lane % lines * 128);
              if (l.res) prefetch_l2(reinterpret_cast<const char*>(static_cast<const TO*>(l.res) + r * l.ldres + f) + lane % lines * 128);
            }
          }
        }
      }
    } else if (warp == 3) {
      // lays the factors of the CTA's tokens and either half's features, kBatch k-blocks to a slot, whose loads are in flight together.  (Asked
      // for by the epilogue's own threads, the loads held up their reads of TMEM: a k-block in four took twice as long.)
      uint32_t at = 0;
      bool ok = true;
      while (ok && walk.next<kForward>(p, tl)) {
        const int fb = min(tl.fti * 2, bp.s.nfb - 1), have = tl.nj - rank * kBM - lane;
        const float* sw = bp.s.w + ((size_t)tl.g * bp.s.nfb + (lane & 1 ? min(fb + 1, bp.s.nfb - 1) : fb)) * l.nk + lane / 2;      // a half and a k-block a lane
        const float* sx = bp.s.x + (int64_t)(tl.row0 + rank * kBM + lane) * bp.s.row;
        for (int left = l.nk; left > 0; left -= kBatch, ++at) {
          float v[kBatch][4];
          const float w = lane < 2 * min(kBatch, left) ? __ldg(sw) : 0.f;
#pragma unroll
          for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[b][i] = b < left && 32 * i < have ? __ldg(sx + b * bp.s.block + i * 32 * bp.s.row) : 0.f;
          sw += kBatch;
          sx += kBatch * bp.s.block;
          const int slot = at % kFactorSlots;
          if (!(ok = __all_sync(0xffffffffu, wait(&s->sempty[slot], ((at / kFactorSlots) & 1) ^ 1, abort_flag)))) break;
#pragma unroll
          for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float f = __shfl_sync(0xffffffffu, w, 2 * b + h);
#pragma unroll
              for (int i = 0; i < 4; ++i) s->factor[slot][b][h][lane + 32 * i] = v[b][i] * f;
            }
          __syncwarp();
          if (lane == 0) mbar_arrive(&s->sfull[slot]);
        }
      }
    }
  } else {
    regs_take<kManyRegs>();
    const int q = warp & 3, half = (warp >> 2) - 1;  // TMEM lanes 32 q ..: 32 tokens; 128 features
    float* turn = reinterpret_cast<float*>(smem + kBlockRing) + (warp - 4) * kTurn;
    const uint32_t tempty0 = mapa(smem_u32(&s->tempty[0]), 0);
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + half * kBM;
    uint32_t n = 0, batch = 0;
    for (uint32_t tiles = 0;; ++tiles) {
      const int slot = tiles % kTileSlots;
      if (!__all_sync(0xffffffffu, wait(&s->told[slot], (tiles / kTileSlots) & 1, abort_flag))) break;
      const volatile int4* tile = &s->tile[slot];
      if (tile->z == 0) break;
      float acc[kBM];
#pragma unroll
      for (int j = 0; j < kBM; ++j) acc[j] = 0.f;
      uint32_t d0 = 0;
      bool ok = true;
      // Few instructions: what a k-block costs beside its multiply-adds, two warps of a scheduler do not hide.
      for (int left = l.nk; left > 0; left -= kBatch, ++batch) {
        const int from = batch % kFactorSlots;
        if (!(ok = __all_sync(0xffffffffu, wait(&s->sfull[from], (batch / kFactorSlots) & 1, abort_flag)))) break;
        const float* factor = &s->factor[from][0][half][32 * q + lane];
        for (int end = left - min(kBatch, left), at = left; at > end; --at, ++n, factor += 2 * kBM) {
          const int buf = n & 1;
          if (!(ok = __all_sync(0xffffffffu, wait<kTmem>(&s->tfull[buf], (n >> 1) & 1, abort_flag)))) break;
          tc_after();
          d0 = lanes + buf * 2 * kBM;
          const float f = *factor;
#pragma unroll
          for (int c = 0; c < kBM; c += 32) {
            float d[32];
            tmem_ld32(d0 + c, d);
            // the buffer is the next k-block's but one's, unless it is the last: then the sums go there
            if (c + 32 == kBM && at > 1) {
              tc_before();
              if (lane == 0) mbar_arrive_relaxed(tempty0 + buf * 8);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[c + j] = fmaf(d[j], f, acc[c + j]);
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s->sempty[from]);
      }
      if (!ok) break;
      // the sums go to the last k-block's buffer, which this warp has read: the registers are the finish's
#pragma unroll
      for (int c = 0; c < kBM; c += 16) {
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = acc[c + j];
        tmem_st16(d0 + c, v);
      }
      const int g = tile->x, first = rank * kBM + 32 * q, row = tile->y + first, f0 = (tile->w * 2 + half) * kBM, rows = tile->z - first;
#pragma unroll 1
      for (int i = 0; i < kBM && f0 + i < l.N && rows > 0; i += 32)
        pair_finish<TO, false, 2>(l, g, row, f0 + i, min(32, rows), 0, turn, [&](auto body) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[16];
            tmem_ld16(d0 + i + 16 * h, v);
#pragma unroll
            for (int j = 0; j < 16; j += 4)          // as [token][32 features], 16-byte chunks at chunk ^ (token & 7)
              *reinterpret_cast<float4*>(turn + lane * 32 + (((4 * h + j / 4) ^ (lane & 7)) * 4)) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          }
          __syncwarp();
          body(0);
          __syncwarp();
          return true;
        });
      tc_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_relaxed(tempty0 + ((n - 1) & 1) * 8);
        mbar_arrive(&s->heard[slot]);
      }
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

// ------------------------------------------------------------------ split kernel

struct BlockSplitParams {
  SplitParams p;
  Scales s;
};

template <int BN> struct BlockSplitTail {
  static constexpr int kMaxStages = 12, kSlots = 4;
  float factor[kSlots][kBatch][BN];
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[4], tempty[4], sfull[kSlots], sempty[kSlots], got;
  uint32_t tmem;
  int abort_flag;
  int g, row0, nj;                  // this cluster's tile; nj = 0: none
};

template <typename TO, int BN>
__global__ void __launch_bounds__(kThreads, 2) linear_blocks_split_kernel(const __grid_constant__ BlockSplitParams sp) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  using Tail = BlockSplitTail<BN>;
  const SplitParams& p = sp.p;
  constexpr int kStage = kABlock + BN * kBKBytes;
  Tail* s = reinterpret_cast<Tail*>(smem + p.stages * kStage);
  volatile int* abort_flag = &s->abort_flag;
  const LinearParams& l = p.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.splits > 1 ? (int)cluster_rank() : 0;
  const int tile = blockIdx.x / p.splits;
  constexpr int kAccs = 4;
  constexpr uint32_t kCols = kAccs * BN < 32 ? 32 : kAccs * BN;

  if (threadIdx.x == 0) {
    prefetch_map(&p.w);
    prefetch_map(&p.x);
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&s->full[i], 1);
      mbar_init(&s->empty[i], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(&s->tfull[i], 1);
      mbar_init(&s->tempty[i], 4);
    }
    for (int i = 0; i < Tail::kSlots; ++i) {
      mbar_init(&s->sfull[i], 1);
      mbar_init(&s->sempty[i], 4);
    }
    mbar_init(&s->got, 1);
    s->abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc<1>(&s->tmem, kCols);
  int g = 0, nj = 0, row0 = tile / p.nft * BN;
  const int fti = tile % p.nft;
  if (!l.offsets) {                                  // dense: the tile is known before the inputs are
    nj = min(BN, l.T - row0);
    tc_before();
    __syncthreads();
    tc_after();
    ops_begin();
  } else {
    ops_begin();
    if (warp == 3) {                                 // token tile tile / nft of the groups' tiles
      const auto tiles = [&](int n) { return (n + BN - 1) / BN; };
      GroupTiles at(tile / p.nft);
      if (at.find(l, tiles)) {
        int n;
        const int t = at.get(tiles, g, row0, n);
        row0 += t * BN;
        nj = min(BN, n - t * BN);
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
  float* own = reinterpret_cast<float*>(smem);       // [token][feature]: the ring is idle by then
  float* got = own + BN * kBM;                       // the other ranks' partials of this rank's share
  const int j0 = nj * rank / p.splits, j1 = nj * (rank + 1) / p.splits;

  if (nj > 0 && warp == 0 && elect()) {
    uint32_t st = 0, phase = 1;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!wait(&s->empty[st], phase, abort_flag)) break;
      const uint32_t a = smem_u32(smem + st * kStage);
      mbar_expect(&s->full[st], kStage);
      tma_3d<1>(a, &p.w, smem_u32(&s->full[st]), kb * kBKBytes, fti * kBM, g);
      tma_2d<1>(a + kABlock, &p.x, smem_u32(&s->full[st]), kb * kBKBytes, row0);
      if (++st == p.stages) st = 0, phase ^= 1;
    }
  } else if (nj > 0 && warp == 1 && elect()) {
    const uint32_t idesc = mma_desc<true>(kBM, BN);
    uint32_t st = 0, phase = 0;
    for (int i = 0; i < kb1 - kb0; ++i) {
      const int buf = i % kAccs;
      if (!wait(&s->tempty[buf], ((i / kAccs) & 1) ^ 1, abort_flag) || !wait(&s->full[st], phase, abort_flag)) break;
      tc_after();
      product_block<1, kForward, true>(tmem + buf * BN, smem_u32(smem + st * kStage), idesc, false, kBoxRows);
      commit<1>(&s->empty[st]);
      commit<1>(&s->tfull[buf]);
      if (++st == p.stages) st = 0, phase ^= 1;
    }
  } else if (nj > 0 && warp == 3) {
    uint32_t at = 0;
    lay_factors<Tail::kSlots, BN>(sp.s, l, g, fti, row0, nj, kb0, kb1, s->factor, s->sfull, at, [&](int slot, uint32_t parity) {
      return __all_sync(0xffffffffu, wait(&s->sempty[slot], parity, abort_flag));
    });
  } else if (nj > 0 && warp >= 4) {
    const int q = warp & 3, row = 32 * q + lane;     // TMEM lane: a feature
    const uint32_t t = tmem + ((uint32_t)(32 * q) << 16);
    float acc[BN];
#pragma unroll
    for (int j = 0; j < BN; ++j) acc[j] = 0.f;
    bool ok = true;
    for (int i = 0; i < kb1 - kb0; ++i) {
      const int buf = i % kAccs, batch = i / kBatch, slot = batch % Tail::kSlots, in = i % kBatch;
      if (in == 0) ok = wait(&s->sfull[slot], (batch / Tail::kSlots) & 1, abort_flag);
      ok = ok && wait(&s->tfull[buf], (i / kAccs) & 1, abort_flag);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;                  // whole warps read TMEM
      tc_after();
      const uint32_t factor = smem_u32(s->factor[slot][in]);
#pragma unroll
      for (int c = 0; c < BN; c += 16)
        if (c < nj) {
          float d[16];
          tmem_ld16(t + buf * BN + c, d);
          take(acc + c, d, factor + 4 * c);
        }
      tc_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_relaxed(smem_u32(&s->tempty[buf]));
        if (in == kBatch - 1) mbar_arrive(&s->sempty[slot]);
      }
    }
    // all warps' last buffers are full: no product reads the ring any more
    if (ok) {
#pragma unroll
      for (int j = 0; j < BN; ++j) own[j * kBM + row] = acc[j];
    }
    if (p.splits > 1) fence_async();
    if (p.splits > 1 && threadIdx.x == 128) mbar_expect(&s->got, (p.splits - 1) * (j1 - j0) * kBM * 4);
  }
  __syncwarp();
  if (p.splits > 1) {
    cluster_sync();                                  // all rings are idle, all partials written
    if (nj > 0 && warp == 0 && lane < p.splits && lane != rank) {
      const int i0 = nj * lane / p.splits, i1 = nj * (lane + 1) / p.splits, share = (i1 - i0) * kBM;
      if (share > 0)
        bulk_to_cluster(mapa(smem_u32(got + rank * share), lane), smem_u32(own + i0 * kBM), share * 4, mapa(smem_u32(&s->got), lane));
    }
    if (nj > 0) wait<kCluster>(&s->got, 0, abort_flag);
  } else {
    __syncthreads();
  }
  if (nj > 0) {                                      // every rank sums and finishes its share of the tokens
    if (l.wide)
      split_finish<TO, 8, false>(p, g, row0, fti * kBM, own, got, rank, j0, j1, threadIdx.x % 16 * 8, 1, threadIdx.x / 16, kThreads / 16);
    else
      split_finish<TO, 4, false>(p, g, row0, fti * kBM, own, got, rank, j0, j1, lane, 32, warp, kThreads / 32);
  }
  settle(abort_flag);
  if (p.splits > 1) cluster_sync();                  // the copies out of a rank's memory have been received
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 2) tmem_dealloc<1>(tmem, kCols);
}

// ------------------------------------------------------------------ few tokens

// As the forward product's kernel for up to 16 tokens: weights straight into the registers of warp-wide matrix instructions.  A warp
// takes whole k-blocks, kBlocks of them in flight, so that their sums stand under one scale a token.  Block (b, i): 8 FS features of up
// to 8 TS tokens, those of the i-th group that has rows; TS or FS is 1.
constexpr int few_blocks(int ts, int fs) { return ts + fs == 2 ? 4 : 2; }
template <typename TO, int TS, int FS>
__global__ void __launch_bounds__(kFewThreads, 1) linear_blocks_few_kernel(const __grid_constant__ FewParams p, const __grid_constant__ Scales sc) {
  constexpr int kBlocks = few_blocks(TS, FS), kFeatures = 8 * FS;
  static_assert(TS * FS <= 2, "one tile of 16 x 8 sums");
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
  const Finish<TO, 1, false> finish(l, g, out ? of : l.N, 1);
  const Place<TO> place(l, row0 + ot, of);
  typename Finish<TO, 1, false>::Ahead ahead;
  finish.ahead(ahead, place, 0, out);

  // rows in units of 16 bytes; a row that does not exist is not read
  const int units = l.F / 16;
  const uint4 *w[FS], *x[TS];
  int wu[FS], xu[TS];
#pragma unroll
  for (int i = 0; i < FS; ++i) {
    const int f = blockIdx.x * kFeatures + i * 8 + lane / 4;
    wu[i] = f < l.N ? units : 0;
    w[i] = static_cast<const uint4*>(p.w) + ((size_t)g * l.N + (f < l.N ? f : 0)) * (p.ldw / 16);
  }
#pragma unroll
  for (int i = 0; i < TS; ++i) {
    const int t = i * 8 + lane / 4;
    xu[i] = t < nt ? units : 0;
    x[i] = static_cast<const uint4*>(p.x) + (row0 + (t < nt ? t : 0)) * (size_t)(p.ldx / 16);
  }
  // the tokens of this lane's sums: features on the instruction's rows (FS = 2), two adjacent columns; else rows 8 apart
  const int t0 = FS == 2 ? lane % 4 * 2 : lane / 4;
  constexpr int kNext = FS == 2 ? 1 : 8;             // from t0 to the second
  const float* sx = sc.x + (int64_t)(row0 + t0) * sc.row;
  const float* sw = sc.w + ((size_t)g * sc.nfb + blockIdx.x * kFeatures / kBM) * l.nk;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  float sum[4] = {};
  for (int b0 = warp; b0 < l.nk; b0 += kBlocks * warps) {
    uint4 wv[FS][kBlocks][2], xv[TS][kBlocks][2];
    float f[kBlocks][2], fw[kBlocks];
#pragma unroll
    for (int u = 0; u < kBlocks; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (b0 + u * warps) * 8 + h * 4 + lane % 4;
#pragma unroll
        for (int i = 0; i < FS; ++i) wv[i][u][h] = k < wu[i] ? __ldcs(w[i] + k) : zero;
      }
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      const int b = b0 + u * warps;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < TS; ++i) xv[i][u][h] = b * 8 + h * 4 + lane % 4 < xu[i] ? __ldg(x[i] + b * 8 + h * 4 + lane % 4) : zero;
      fw[u] = b < l.nk ? __ldg(sw + b) : 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) f[u][j] = b < l.nk && t0 + kNext * j < nt ? __ldg(sx + kNext * j * sc.row + b * sc.block) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      float c[4] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (FS == 2)
          warp_mma<true>(c, wv[0][u][h], wv[1][u][h], xv[0][u][h]);
        else
          warp_mma<true>(c, xv[0][u][h], TS == 2 ? xv[TS - 1][u][h] : zero, wv[0][u][h]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float s = f[u][FS == 2 ? j % 2 : j / 2] * fw[u];
        if (b0 + u * warps < l.nk) sum[j] = fmaf(c[j], s, sum[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = lane / 4 + j / 2 * 8, q = lane % 4 * 2 + j % 2;
    if (FS == 2) part[warp][q * kFeatures + r] = sum[j];
    else if (TS == 2 || j < 2) part[warp][r * kFeatures + q] = sum[j];
  }
  __syncthreads();
  if (out) {
    float v[1] = {part[0][threadIdx.x]};
    for (int i = 1; i < warps; ++i) v[0] += part[i][threadIdx.x];
    finish(v, place.y, ahead);
  }
}

// ------------------------------------------------------------------ quantisers

constexpr float kE4M3Max = 448.f;
constexpr int kQuantBlock = 128;

// The scale of a block whose largest |value| has these bits (NaN above infinity), and quotients by it that round as a division's do
// wherever e4m3 can tell (below 2^-11 all become zeros).  1 / scale = hi + lo to 2^-47: hi is the rounded one, lo the rest.  v (hi + lo), as
// v hi + round(v lo) rounded once, is a neighbour of v / scale in fp32.
// fp32: from there one exact remainder gives the rounded quotient (Markstein, IBM J. Res. Dev. 34 (1990) 111).
// bf16: it is the rounded quotient itself, unless that lies within 2^-46 of the middle between two fp32 numbers, which e4m3 can tell only
// next to a border C between two of its numbers (five bits).  There v would be C (1 + 2^-24) scale or so to 46 bits; but scale is a bf16 number's
// 448th part, eight bits or a seventh's repeating ones, whose products with that end in no 20 zeros (tests try every pair of mantissas).
// v times 1 / scale alone, two roundings, moved 5e-4 of the elements to the next number: exact ties are common, since 448 = 7 * 64.
// One element at a time these steps took 2.7 us more of 4096 x 7168 and 3.4 of 8 x 2048 x 7168 than that product, two at a time nothing.
template <typename T> struct Divisor {
  float scale, by, hi, lo, shift;
  __device__ __forceinline__ explicit Divisor(uint32_t bits) {
    scale = fmaxf(__fdiv_rn(__uint_as_float(bits), kE4M3Max), 1.17549435e-38f);
    if (bits >= 0x7f800000u) scale = __uint_as_float(0x7fffffffu);       // an infinity or a NaN: all of the block is NaN
    shift = scale > 0x1p64f ? 0x1p-64f : scale < 0x1p-64f ? 0x1p64f : 1.f;         // lo and the remainders stay normal numbers
    by = scale * shift;
    hi = __frcp_rn(by);
    lo = fmaf(-hi, by, 1.f) * hi;
  }
  // the divisor of lane `src` of this lane's four, by whole warps; SHIFTS: shifts are other than 1 somewhere in the warp
  __device__ __forceinline__ Divisor(const Divisor& d, int src, bool shifts) {
    hi = __shfl_sync(0xffffffffu, d.hi, src, 4);
    lo = __shfl_sync(0xffffffffu, d.lo, src, 4);
    if (sizeof(T) == 4) by = __shfl_sync(0xffffffffu, d.by, src, 4);
    shift = shifts ? __shfl_sync(0xffffffffu, d.shift, src, 4) : 1.f;
  }
  __device__ __forceinline__ void divide(float (&v)[8]) const {
    if (shift != 1.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= shift;
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2) {                 // two at a time
      float2 w = make_float2(v[i], v[i + 1]);
      const float2 hh = make_float2(hi, hi), q = __ffma2_rn(w, hh, __fmul2_rn(w, make_float2(lo, lo)));
      w = sizeof(T) == 2 ? q : __ffma2_rn(__ffma2_rn(make_float2(-q.x, -q.y), make_float2(by, by), w), hh, q);
      v[i] = w.x, v[i + 1] = w.y;
    }
  }
};

__device__ __forceinline__ uint32_t largest(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// 8 elements of a row from column c, as they lie in memory; those at `width` and behind are zeros.  WIDE: in 16-byte units.
template <typename T, bool WIDE> struct Eight {
  T v[8];
  __device__ __forceinline__ void load(const T* row, int64_t c, int64_t width) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < width ? row[c + i] : from_f<T>(0.f);
  }
  __device__ __forceinline__ void get(float (&t)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = to_f(v[i]);
  }
  __device__ __forceinline__ uint32_t most() const {
    float t[8];
    get(t);
    return largest(t);
  }
};
template <typename T> struct Eight<T, true> {
  static constexpr int N = Vec<T>::N;
  uint4 v[8 / N];
  __device__ __forceinline__ void load(const T* row, int64_t c, int64_t width) {
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) v[i] = c < width ? __ldg(reinterpret_cast<const uint4*>(row + c) + i) : make_uint4(0, 0, 0, 0);   // width: a multiple of 8
  }
  // the bits of the largest |value|, as fp32 (NaN above infinity): two at a time in 16 bits
  __device__ __forceinline__ uint32_t most() const {
    if constexpr (N == 8) {
      __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v[0].x));
      m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v[0].y)));
      m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v[0].z)));
      m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v[0].w)));
      return (uint32_t)__bfloat16_as_ushort(__hmax_nan(m.x, m.y)) << 16;
    } else {
      float t[8];
      get(t);
      return largest(t);
    }
  }
  __device__ __forceinline__ void get(float (&t)[8]) const {
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) {
      float u[N];
      unpack16<T>(v[i], u);
#pragma unroll
      for (int j = 0; j < N; ++j) t[i * N + j] = u[j];
    }
  }
};
template <bool WIDE>
__device__ __forceinline__ void store8(uint8_t* row, int64_t c, int64_t width, const float (&v)[8]) {
  if constexpr (WIDE) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3) |
             (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
    if (c < width) *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < width) row[c + i] = __nv_cvt_float_to_fp8(v[i], __NV_SATFINITE, __NV_E4M3);
  }
}
template <typename T> struct QuantParams {
  Rows<const T> x;
  Rows<uint8_t> q;
  float* scale;
  int64_t scale_row, scale_block, rows, width;
  int blocks;                       // of 128 columns
};

// 1 x 128: sixteen lanes take a block of a row, 8 elements each; a thread asks for kU blocks before it uses the first.  A block of
// threads takes kU * 16 blocks of 128 side by side of kRows rows, so that neither needs a division; the scales of a column of blocks,
// whose rows lie side by side, are written kRows at a time.
constexpr int kQuantRows = 8;                        // 4096 x 7168 in bf16 17.1 us; with 4 a microsecond more
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantParams<T> p) {
  constexpr int kU = 4, kRows = kQuantRows;          // blocks of a thread; rows of a block of threads
  ops_begin();
  const int sub = threadIdx.x / 16, at = threadIdx.x % 16 * 8;
  const int64_t row = (int64_t)blockIdx.y * kRows + sub % kRows + (int64_t)blockIdx.z * 65535 * kRows;
  const int first = blockIdx.x * (kU * 16 / kRows) + sub / kRows;
  Eight<T, WIDE> x[kU];
  if (row < p.rows) {
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (first + u * (16 / kRows) < p.blocks) x[u].load(p.x.at(row), (int64_t)(first + u * (16 / kRows)) * kQuantBlock + at, p.width);
  }
  // a divisor takes some 30 instructions: of each four lanes, one works out each of the four blocks' for the others
  static_assert(kU == 4, "a block's divisor a lane");
  uint32_t bits = 0;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    uint32_t m = row < p.rows && first + u * (16 / kRows) < p.blocks ? x[u].most() : 0;
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (threadIdx.x % kU == u) bits = m;
  }
  const Divisor<T> mine(bits);
  const bool shifts = __any_sync(0xffffffffu, mine.shift != 1.f);
  const int my_col = first + threadIdx.x % kU * (16 / kRows);
  if (threadIdx.x % 16 < kU && row < p.rows && my_col < p.blocks) p.scale[row * p.scale_row + my_col * p.scale_block] = mine.scale;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const Divisor<T> by(mine, u, shifts);
    const int col = first + u * (16 / kRows);
    if (row >= p.rows || col >= p.blocks) continue;
    float v[8];
    x[u].get(v);
    by.divide(v);
    store8<WIDE>(p.q.at(row), (int64_t)col * kQuantBlock + at, p.width, v);
  }
}

// 128 x 128: a block of 256 threads takes a block of the matrix, which stays in its registers, as it was read, between maximum and
// quotient.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256, WIDE && sizeof(T) == 2 ? 4 : 2) quantize_weight_kernel(const QuantParams<T> p) {
  __shared__ uint32_t part[8];
  ops_begin();
  constexpr int kRows = kQuantBlock / 16;            // of a thread
  const int sub = threadIdx.x / 16;
  const int64_t row0 = (int64_t)blockIdx.y * kQuantBlock, g = blockIdx.z, c = (int64_t)blockIdx.x * kQuantBlock + threadIdx.x % 16 * 8;
  Eight<T, WIDE> v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)                    // a row behind the last is the last one again
    v[i].load(p.x.at(g * p.rows + min(row0 + sub + 16 * i, p.rows - 1)), c, p.width);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) m = max(m, v[i].most());
  m = __reduce_max_sync(0xffffffffu, m);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, part[i]);
  const Divisor<T> by(m);
  if (threadIdx.x == 0) p.scale[(g * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = by.scale;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (row0 + sub + 16 * i >= p.rows) continue;
    float t[8];
    v[i].get(t);
    by.divide(t);
    store8<WIDE>(p.q.at(g * p.rows + row0 + sub + 16 * i), c, p.width, t);
  }
}

// ------------------------------------------------------------------ host side

template <typename TO>
moe_status launch_pair(const moe_async_linear_args* a, const LinearParams& l, const Scales& sc, int sms, void* s) {
  // the warps wait for registers that the launch does not have if the compiler gave it fewer
  static const bool fits = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, linear_blocks_pair_kernel<TO>) == cudaSuccess && at.numRegs >= kLaunchRegs;
  }();
  if (!fits) return MOE_ERR_CUDA;
  BlockPairParams b;
  PairParams& p = b.p;
  b.s = sc;
  p.l = l;
  p.nft = (l.N + 2 * kBM - 1) / (2 * kBM);
  if (!encode(&p.w, a->d_w, 1, l.F, l.N, a->w_stride, l.G, kBM)) return MOE_ERR_CUDA;
  p.tokens = 2 * kBM;
  if (!encode(&p.x[3], a->d_x, 1, l.F, l.T, a->x_stride, 0, kBM)) return MOE_ERR_CUDA;
  if (cudaFuncSetAttribute(linear_blocks_pair_kernel<TO>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBlockPairSmem) != cudaSuccess) return MOE_ERR_CUDA;
  return launch_op(linear_blocks_pair_kernel<TO>, dim3(sms / 2 * 2), kPairThreads, kBlockPairSmem, 1, s, b);
}

template <int BN>
constexpr int block_split_stages(bool own_sm) {
  const int n = ((own_sm ? kSplitSmem : kSplitSmem / 2) - (int)sizeof(BlockSplitTail<BN>) - 1024) / (kABlock + BN * kBKBytes);
  return n < BlockSplitTail<BN>::kMaxStages ? n : BlockSplitTail<BN>::kMaxStages;
}

int blocks_split_capacity(int s, int sms) {
  static Capacities known;
  return s == 1 ? sms : capacity_of(linear_blocks_split_kernel<__nv_bfloat16, 64>, known, s, sms);
}

template <typename TO, int BN>
moe_status launch_split(const moe_async_linear_args* a, const LinearParams& l, const Scales& sc, int sms, int splits, int64_t tiles, void* s) {
  // the ring holds the CTA's partials and its share of up to 8 ranks' (which may round up by a token each)
  static_assert((BN + BN + 8) * kBM * 4 <= block_split_stages<BN>(false) * (kABlock + BN * kBKBytes), "shared memory of the split kernel");
  BlockSplitParams b;
  SplitParams& p = b.p;
  b.s = sc;
  p.l = l;
  p.bn = BN;
  p.splits = splits;
  p.nft = (l.N + kBM - 1) / kBM;
  // where clusters of whole-SM CTAs do not all find a place, two share an SM (148 CTAs in clusters of 4, 64 x 7168 x 4736: 14.9 us, alone 22.6)
  p.stages = block_split_stages<BN>(tiles * splits <= blocks_split_capacity(splits, sms) && l.nk > block_split_stages<BN>(false) * splits);
  const int smem = p.stages * (kABlock + BN * kBKBytes) + (int)sizeof(BlockSplitTail<BN>) + 1024;
  if (!encode(&p.w, a->d_w, 1, l.F, l.N, a->w_stride, l.G, kBM) || !encode(&p.x, a->d_x, 1, l.F, l.T, a->x_stride, 0, BN)) return MOE_ERR_CUDA;
  if (cudaFuncSetAttribute(linear_blocks_split_kernel<TO, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmem) != cudaSuccess) return MOE_ERR_CUDA;
  return launch_op(linear_blocks_split_kernel<TO, BN>, dim3((unsigned)(tiles * splits)), kThreads, smem, splits, s, b);
}

template <typename TO, int TS, int FS>
moe_status launch_few(const moe_async_linear_args* a, const LinearParams& l, const Scales& sc, void* s) {
  const FewParams p{a->d_x, a->d_w, a->x_stride, a->w_stride, l};
  const dim3 grid((unsigned)((l.N + 8 * FS - 1) / (8 * FS)), (unsigned)(l.offsets ? std::min(l.G, l.T) : 1));
  // half the warps where these take K in one pass all the same
  const int threads = l.nk <= few_blocks(TS, FS) * (kFewThreads / 64) ? kFewThreads / 2 : kFewThreads;
  return launch_op(linear_blocks_few_kernel<TO, TS, FS>, grid, threads, 0, 1, s, p, sc);
}

// Kernel, tile and split with the least expected time, in ns, from 25 shapes of 17 to 4096 tokens on 256 to 7168 features, dense and in 32
// to 128 groups.  A k-block costs a split CTA of 16, 32 or 64 tokens 200, 260 or 360 alone on its SM, 330, 400 or 560 beside another; a
// pair 430 in its first tile, 480 in those after, with 3,300 for the finish between.  The exchange takes 350 to 720 a rank.  `bytes`: all
// operands; of the smaller of stream and sums, part shows.  Groups count half a tile each for their ends.
// The choice's time is 4% above the best one's on average, 45% at worst (64 tokens on 7168 x 256: 10.5 against 7.2).
LinearPlan blocks_plan(const LinearParams& l, int sms, float bytes) {
  const float groups = l.offsets ? std::min(l.G, l.T) : 1, per = l.T / groups;
  const auto token_tiles = [&](int t) { return l.offsets ? std::max(groups, l.T / (float)t + 0.5f * groups) : (float)((l.T + t - 1) / t); };
  LinearPlan plan{false, 64, 1};
  float best = 1e30f;
  for (int bn = per <= 16 ? 16 : per <= 32 ? 32 : 64; bn <= 64; bn *= 2)
    for (int s = 1; s <= 8 && (s == 1 || 2 * s <= l.nk); s *= 2) {
      const float ctas = (l.N + kBM - 1) / kBM * token_tiles(bn) * s, own = (float)blocks_split_capacity(s, sms);
      const float waves = std::max(1.f, l.offsets ? ctas / (2 * own) : std::ceil(ctas / (2 * own)));
      const bool alone = ctas <= own;
      const float kb = (l.nk + s - 1) / s * (bn == 16 ? alone ? 200.f : 330.f : bn == 32 ? alone ? 260.f : 400.f : alone ? 360.f : 560.f);
      const float ns = (s == 1 ? 3600.f : 3900.f + (bn == 64 ? 720.f : 350.f) * s) + kb + (waves - 1) * (kb + 2500.f);
      if (ns < best) best = ns, plan.tokens = bn, plan.splits = s;
    }
  const float stream = 4000.f + bytes / 6400.f;
  best = std::max(best, stream) + 0.15f * std::min(best, stream);
  const float rounds = (l.N + 2 * kBM - 1) / (2 * kBM) * token_tiles(2 * kBM) / (sms / 2);
  float ns = 7200.f + 430.f * l.nk + std::max(0.f, std::ceil(rounds) - 1.f) * (480.f * l.nk + 3300.f);
  ns = std::max(ns, 5500.f + bytes / 5500.f) + 0.05f * ns;
  if (ns < best) plan = {true, 2 * kBM, 1};
  return plan;
}

template <typename TO>
moe_status blocks_launch(const moe_async_linear_args* a, const LinearParams& l, const Scales& sc, void* s) {
  const int sms = sm_count();
  if (sms < 2) return MOE_ERR_CUDA;
  const int groups = l.offsets ? std::min(l.G, l.T) : 1;
  // Up to 8 tokens the few kernel is ahead on small weights, to the forward product's bounds (few / split us, 1 and 8 tokens: on 512 x 256
  // 3.6 / 4.6, 2880 x 2880 5.6 / 6.6, 7168 x 2048 5.8 / 8.3, 2048 x 9728 6.6 / 8.4, 7168 x 4096 9.8 / 9.9 and 10.1 / 10.1; beyond them 7168 x
  // 7168 14.5 / 13.1, 512 x 16384 7.0 / 4.9, 8 rows of 32 groups on 7168 x 2048 32 / 24).  For 16 it holds one k-block in flight where it takes
  // 16 features a block: 2880 x 2880 7.7 / 6.9, 2048 x 9728 11.4 / 8.5, 7168 x 4096 14.0 / 10.1 (7168 x 2048 8.0 / 8.5); with 8 features 7168
  // x 256 4.8 / 7.2, 7168 x 1024 5.6 / 8.0.
  const int64_t features = (int64_t)l.N * groups;
  const bool wide_rows = features > 8 * sms;         // 16 features a block
  if (l.T <= kFewTokens && features <= 64 * sms && features * l.F <= 32'000'000 && !(l.T > 8 && wide_rows))
    return l.T > 8 ? launch_few<TO, 2, 1>(a, l, sc, s) : wide_rows ? launch_few<TO, 1, 2>(a, l, sc, s) : launch_few<TO, 1, 1>(a, l, sc, s);
  const LinearPlan plan = blocks_plan(l, sms, ((float)features + l.T) * l.F);
  if (plan.pair) return launch_pair<TO>(a, l, sc, sms, s);
  const int64_t tiles = (int64_t)((l.N + kBM - 1) / kBM) * (l.offsets ? l.T / plan.tokens + groups : (l.T + plan.tokens - 1) / plan.tokens);
  return plan.tokens == 16   ? launch_split<TO, 16>(a, l, sc, sms, plan.splits, tiles, s)
         : plan.tokens == 32 ? launch_split<TO, 32>(a, l, sc, sms, plan.splits, tiles, s)
                             : launch_split<TO, 64>(a, l, sc, sms, plan.splits, tiles, s);
}

template <typename T>
moe_status quantize(const void* x, int64_t ldx, int32_t G, int32_t rows, int32_t width, void* q, int64_t ldq, float* scale, int64_t sr, int64_t sb, bool weight,
                    void* s) {
  QuantParams<T> p{{static_cast<const T*>(x), ldx}, {static_cast<uint8_t*>(q), ldq}, scale, sr, sb, rows, width, (int)(((int64_t)width + kQuantBlock - 1) / kQuantBlock)};
  const bool wide = width % 8 == 0 && rows16(x, ldx, sizeof(T)) && reinterpret_cast<uintptr_t>(q) % 8 == 0 && ldq % 8 == 0;
  if (weight) {
    const int64_t rb = ((int64_t)rows + kQuantBlock - 1) / kQuantBlock;
    if (rb > 65535 || G > 65535) return MOE_ERR_UNSUPPORTED;
    return launch_op(wide ? quantize_weight_kernel<T, true> : quantize_weight_kernel<T, false>, dim3((unsigned)p.blocks, (unsigned)rb, (unsigned)G), 256, 0, 1, s, p);
  }
  const int64_t y = ((int64_t)rows + kQuantRows - 1) / kQuantRows;
  const dim3 grid((unsigned)((p.blocks + 7) / 8), (unsigned)std::min<int64_t>(y, 65535), (unsigned)((y + 65534) / 65535));
  return launch_op(wide ? quantize_rows_kernel<T, true> : quantize_rows_kernel<T, false>, grid, 256, 0, 1, s, p);
}

}  // namespace

unsigned int* ops_error_blocks() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_ops_error) == cudaSuccess ? static_cast<unsigned int*>(p) : nullptr;
}

}  // namespace moe

extern "C" moe_status moe_async_linear_blocks(const moe_async_linear_args* a, int64_t x_scale_row, int64_t x_scale_block, void* stream) {
  using namespace moe;
  if (!a) return MOE_ERR_INVALID;
  if (a->rows < 0 || a->rows > INT32_MAX - 1024 || a->fan_in < 1 || a->fan_in > INT32_MAX - 1024 ||
      a->fan_out < 1 || a->fan_out > INT32_MAX - 1024 || a->groups < 0 || a->groups > kMaxExperts ||
      a->act < MOE_ACT_NONE || a->act > MOE_ACT_RELU || (a->groups > 0) != (a->d_offsets != nullptr) ||
      (a->out_dtype != MOE_F32 && a->out_dtype != MOE_BF16) || x_scale_row < 0 || x_scale_block < 0)
    return MOE_ERR_INVALID;
  if (a->dtype != MOE_E4M3) return MOE_ERR_UNSUPPORTED;
  if (a->rows == 0) return MOE_OK;
  if (!a->d_x || !a->d_w || !a->d_y || !a->d_x_scale || !a->d_w_scale || a->x_stride < a->fan_in || a->w_stride < a->fan_in || a->y_stride < a->fan_out ||
      (a->d_mul && a->mul_stride < a->fan_out) || (a->d_residual && a->residual_stride < a->fan_out))
    return MOE_ERR_INVALID;
  // the operands move in 16-byte units
  if (a->fan_in % 16 || !rows16(a->d_x, a->x_stride, 1) || !rows16(a->d_w, a->w_stride, 1)) return MOE_ERR_UNSUPPORTED;
  const int os = dtype_size(a->out_dtype);
  const bool wide = a->fan_out % 8 == 0 && rows16(a->d_y, a->y_stride, os) && rows16(a->d_mul, a->mul_stride, os) &&
                    rows16(a->d_residual, a->residual_stride, os);
  const LinearParams l{a->d_bias,     nullptr,     nullptr,      a->d_mul,   a->d_residual, a->d_y,
                       a->d_offsets,  a->mul_stride, a->residual_stride, a->y_stride, a->rows, a->fan_out,
                       a->fan_in,     std::max(1, a->groups), a->act, (a->fan_in + kBKBytes - 1) / kBKBytes, wide};
  const Scales sc{a->d_x_scale, a->d_w_scale, x_scale_row, x_scale_block, (a->fan_out + kBM - 1) / kBM};
  return a->out_dtype == MOE_BF16 ? blocks_launch<__nv_bfloat16>(a, l, sc, stream) : blocks_launch<float>(a, l, sc, stream);
}

extern "C" moe_status moe_async_quantize_blocks(int32_t dtype, const void* d_x, int64_t x_stride, int32_t G, int32_t rows, int32_t width, int32_t block_rows,
                                                void* d_q, int64_t q_stride, float* d_scale, int64_t scale_row, int64_t scale_block, void* stream) {
  using namespace moe;
  if (rows < 0 || width < 1 || width > kMaxWidth || (block_rows != 1 && block_rows != kQuantBlock) || G < 1 || (block_rows == 1 && G != 1) ||
      (dtype != MOE_F32 && dtype != MOE_BF16))
    return MOE_ERR_INVALID;
  if (rows == 0) return MOE_OK;
  if (!d_x || !d_q || !d_scale || x_stride < width || q_stride < width || scale_row < 0 || scale_block < 0) return MOE_ERR_INVALID;
  return dtype == MOE_F32 ? quantize<float>(d_x, x_stride, G, rows, width, d_q, q_stride, d_scale, scale_row, scale_block, block_rows != 1, stream)
                          : quantize<__nv_bfloat16>(d_x, x_stride, G, rows, width, d_q, q_stride, d_scale, scale_row, scale_block, block_rows != 1, stream);
}
