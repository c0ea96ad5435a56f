// Gradients of the product y[t, n] = sum_f x[t, f] w[n, f], dense or per expert on sorted rows, of the
// product's epilogue act(z) * mul, and of its bias:
//
//   grad_x[t, f]    = sum_n grad[t, n] w[n, f] (+ residual[t, f])
//   grad_w[g, n, f] = sum_t grad[t, n] x[t, f] (+ old)      over the rows t of group g
//   grad_b[g, n]    = sum_t grad[t, n] (+ old)
//
// Both products run on the forward product's kernels (moe_linear.cuh): w lies across grad_x's sum, and both
// operands of grad_w across its own, so the operands stay as they lie in memory and the tensor cores read them
// transposed.  grad_w's sum is as long as the group has rows: its last k-block is filled up with zeros.
#include "moe_linear.cuh"

namespace moe {
namespace {

template <typename TO, int MODE>
moe_status launch_pair(PairArgs<MODE>& p, const LinearParams& l, int tokens, int sms, void* s) {
  constexpr int kSmem = kPairRing + kStaging + (int)sizeof(PairTail) + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  p.l = l;
  p.nft = (l.N + 2 * kBM - 1) / (2 * kBM);
  p.tokens = tokens;
  p.ntt = (l.T + tokens - 1) / tokens;
  p.by_band = Divide::by(8 * p.nft, (int64_t)p.ntt * p.nft);
  p.by_last = Divide::by(std::max(1, p.ntt % 8), 8 * p.nft);
  p.stage_bytes = kABlock + tokens / 2 * kBKBytes;
  p.stages = std::min(PairTail::kMaxStages, pair_ring(MODE) / p.stage_bytes);
  if (cudaFuncSetAttribute(linear_pair_kernel<false, TO, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
    return MOE_ERR_CUDA;
  return launch_op(linear_pair_kernel<false, TO, MODE>, dim3(sms / 2 * 2), kPairThreads, kSmem, 1, s, p);
}

template <typename TO, int MODE>
moe_status launch_split(SplitParams& p, const LinearParams& l, int bn, int splits, int64_t tiles, int sms, void* s) {
  p.l = l;
  p.bn = bn;
  p.splits = splits;
  p.nft = (l.N + kBM - 1) / kBM;
  p.ntt = (l.T + bn - 1) / bn;
  p.stages = split_stages(bn, false);
  if (bn > 64 || (tiles * splits <= split_capacity<MODE>(splits, sms) && l.nk > p.stages * splits)) p.stages = split_stages(bn, true);
  const int smem = p.stages * (kABlock + bn * kBKBytes) + (int)sizeof(SplitTail) + 1024;
  if (cudaFuncSetAttribute(linear_split_kernel<false, TO, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmem) != cudaSuccess)
    return MOE_ERR_CUDA;
  return launch_op(linear_split_kernel<false, TO, MODE>, dim3((unsigned)(tiles * splits)), kThreads, smem, splits, s, p);
}

using Args = moe_async_linear_backward_args;

// grad_x: the forward product's tiles and choice, with w across K.
template <typename TO>
moe_status rows_grad(const Args* a, const void* grad, int64_t grad_stride, int sms, void* s) {
  const bool wide = a->fan_in % 8 == 0 && rows16(a->d_grad_x, a->grad_x_stride, sizeof(TO)) && rows16(a->d_residual, a->residual_stride, sizeof(TO));
  const LinearParams l{nullptr, nullptr, nullptr, nullptr, a->d_residual, a->d_grad_x, a->d_offsets, 0, a->residual_stride, a->grad_x_stride,
                       a->rows, a->fan_in, a->fan_out, std::max(1, a->groups), MOE_ACT_NONE, (int)(((int64_t)a->fan_out * 2 + kBKBytes - 1) / kBKBytes), wide};
  const int groups = l.offsets ? std::min(l.G, l.T) : 1;
  const LinearPlan plan = linear_plan<false, TO, kRowsGrad>(l, sms, ((float)l.N * groups + l.T) * l.F * 2);
  if (plan.pair) {
    PairParams p;
    if (!encode(&p.w, a->d_w, 2, l.N, l.F, a->w_stride, l.G, kBoxRows)) return MOE_ERR_CUDA;
    for (int i = 0; i < 4; ++i)
      if (!encode(&p.x[i], grad, 2, l.F, l.T, grad_stride, 0, i < 3 ? 16 << i : plan.tokens / 2)) return MOE_ERR_CUDA;
    return launch_pair<TO, kRowsGrad>(p, l, plan.tokens, sms, s);
  }
  SplitParams p;
  if (!encode(&p.w, a->d_w, 2, l.N, l.F, a->w_stride, l.G, kBoxRows) || !encode(&p.x, grad, 2, l.F, l.T, grad_stride, 0, plan.tokens))
    return MOE_ERR_CUDA;
  const int64_t tiles = (int64_t)((l.N + kBM - 1) / kBM) * (l.offsets ? l.T / plan.tokens + groups : (l.T + plan.tokens - 1) / plan.tokens);
  return launch_split<TO, kRowsGrad>(p, l, plan.tokens, plan.splits, tiles, sms, s);
}

// Kernel, tile and split of grad_w with the least expected time, in ns, from 20 shapes of 64 to 16384 rows on 208 to 7168 features, dense
// and in 8 to 128 groups (9% above the best one's on average, 28% at worst).  A k-block of 64 rows costs a split CTA of 64 or 128 of fan_out
// 200 or 230 alone on its SM, 310 beside another; a pair 215 in fp32 (128 of fan_out), 270 in bf16 (256).  Which group has how many
// rows is not known here: the average, and half a k-block for its end.
template <typename TO>
LinearPlan weight_plan(const LinearParams& l, int sms) {
  constexpr bool kSums = sizeof(TO) == 4;
  const float nk = l.F / (64.f * l.G) + (l.offsets ? 0.5f : 0.f);
  const auto tiles = [&](int features, int t) { return (float)((l.N + features - 1) / features) * ((l.T + t - 1) / t) * l.G; };
  const float rounds = std::ceil(tiles(2 * kBM, kPairTokens<TO>) / (sms / 2)), kb = (kSums ? 215.f : 270.f) * nk;
  float best = 6500.f + kb + (rounds - 1.f) * (kb + (kSums ? 1300.f : 2000.f));
  LinearPlan plan{true, kPairTokens<TO>, 1};
  for (int bn = 64; bn <= 128; bn *= 2)
    for (int s = 1; s <= 8 && (s == 1 || 2 * s <= nk); s *= 2) {
      const float ctas = tiles(kBM, bn) * s, own = s == 1 ? (float)sms : (float)split_capacity<kWeightGrad>(s, sms);
      const bool alone = ctas <= own;
      // a group may have all rows, and an fp32 sum has four chunks
      if ((!alone && (s > 1 || bn == 128)) || (kSums && (l.F + kBoxRows - 1) / kBoxRows > 4 * kChunkBlocks * s)) continue;
      const float k = nk / s * (!alone ? 310.f : bn == 64 ? 200.f : 230.f);
      const float ns = 4600.f + (s > 1 ? 480.f * s : 0.f) + (bn == 128 ? 1200.f : 0.f) + k + (std::ceil(ctas / (2 * own)) - 1.f) * (k + 4300.f);
      if (ns < best) best = ns, plan = {false, bn, s};
    }
  return plan;
}

template <typename TO>
moe_status weight_grad(const Args* a, const void* grad, int64_t grad_stride, bool beside, int sms, void* s) {
  const bool wide = a->fan_in % 8 == 0 && rows16(a->d_grad_w, a->grad_w_stride, sizeof(TO));
  const LinearParams l{nullptr, nullptr, nullptr, nullptr, a->accumulate ? a->d_grad_w : nullptr, a->d_grad_w, a->d_offsets, 0,
                       a->grad_w_stride, a->grad_w_stride, a->fan_out, a->fan_in, a->rows, std::max(1, a->groups), MOE_ACT_NONE,
                       (a->rows + kBoxRows - 1) / kBoxRows, wide, beside};
  const LinearPlan plan = weight_plan<TO>(l, sms);
  const int64_t tiles = (int64_t)((l.N + kBM - 1) / kBM) * ((l.T + plan.tokens - 1) / plan.tokens) * l.G;
  if (!plan.pair) {
    SplitParams p;
    if (!encode(&p.w, a->d_x, 2, a->fan_in, a->rows, a->x_stride, 0, kBoxRows) || !encode(&p.x, grad, 2, a->fan_out, a->rows, grad_stride, 0, kBoxRows))
      return MOE_ERR_CUDA;
    return launch_split<TO, kWeightGrad>(p, l, plan.tokens, plan.splits, tiles, sms, s);
  }
  AcrossParams p;
  if (!encode(&p.w, a->d_x, 2, a->fan_in, a->rows, a->x_stride, 0, kBoxRows) || !encode(&p.x[0], grad, 2, a->fan_out, a->rows, grad_stride, 0, kBoxRows))
    return MOE_ERR_CUDA;
  for (int i = 0; l.offsets && i < 2; ++i) {
    const void* of = i == 0 ? a->d_x : grad;
    const int width = i == 0 ? a->fan_in : a->fan_out;
    const int64_t ld = i == 0 ? a->x_stride : grad_stride;
    if (!encode(&p.slab[i], of, 2, width, a->rows, ld, 0, 16) || !encode(&p.row[i], of, 2, width, a->rows, ld, 0, 1) ||
        (a->rows >= kBoxRows && !encode_windows(&p.window[i], of, width, a->rows, ld)))
      return MOE_ERR_CUDA;
  }
  p.boxed = wide;                                    // unless rows start off 16-byte boundaries
  if (p.boxed && !encode_result<TO>(&p.y, a->d_grad_w, a->fan_in, a->fan_out, a->grad_w_stride, l.G)) return MOE_ERR_CUDA;
  return launch_pair<TO, kWeightGrad>(p, l, plan.tokens, sms, s);
}

// ------------------------------------------------------------------ the bias's gradient

constexpr int kBiasThreads = 256;
constexpr int kBiasCols = 64;                        // columns of a block: 8 a lane, four rows a warp
constexpr int kBiasAhead = 8, kBiasRanks = 8;        // rows of a lane in flight; CTAs that share a group's rows, at most
// Rows are counted in 32 bits, and the walk over them ends up to this far behind the last one.
constexpr int kBiasStep = kBiasRanks * (kBiasThreads / 32) * 4 * kBiasAhead;
constexpr int kMaxRows = INT32_MAX - 4096;
static_assert((int64_t)kMaxRows + 2 * kBiasStep <= INT32_MAX && (int64_t)kMaxRows + 1024 <= INT32_MAX, "the bias's rows, and the products' tiles");

// Column sums of a group's rows, bound by their one read.  A cluster takes 64 columns of a group (128 bytes a row; 256 columns left 2048 x
// 256 to eight CTAs, 6.2 us): every quarter of its warps each so-many-th row, eight loads in flight.  Quarters meet by shuffles, warps in
// shared memory, CTAs in the first one's, all in a fixed order.
__global__ void __launch_bounds__(kBiasThreads)
    grad_bias_kernel(const __nv_bfloat16* __restrict__ grad, int64_t ld, const LinearParams l, float* __restrict__ out, int add) {
  __shared__ float part[kBiasThreads / 32][kBiasCols];
  if (l.beside) ops_beside();
  else ops_begin();
  const int ranks = (int)cluster_size(), rank = (int)cluster_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = kBiasThreads / 32;
  const int blocks = (l.T + kBiasCols - 1) / kBiasCols, at = blockIdx.x / ranks;
  const int g = at / blocks, c = at % blocks * kBiasCols + lane % 8 * 8;
  const Span sp = group_rows(l, g, l.F);
  float v[8] = {};
  const int step = ranks * warps * 4, first = (rank * warps + warp) * 4 + lane / 8;
  if (c + 8 <= l.T) {
    constexpr int kAt = kBiasAhead;
    for (int r = first; r < sp.n; r += kAt * step) {
      uint4 u[kAt];
#pragma unroll
      for (int i = 0; i < kAt; ++i)
        u[i] = r + i * step < sp.n ? __ldg(reinterpret_cast<const uint4*>(grad + (int64_t)(sp.a + r + i * step) * ld + c)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        float t[8];
        unpack16<__nv_bfloat16>(u[i], t);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += t[j];
      }
    }
  } else {
    for (int r = first; r < sp.n; r += step)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < l.T) v[j] += __bfloat162float(grad[(int64_t)(sp.a + r) * ld + c + j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] += __shfl_xor_sync(0xffffffffu, v[j], 8);
    v[j] += __shfl_xor_sync(0xffffffffu, v[j], 16);
    if (lane < 8) part[warp][lane * 8 + j] = v[j];
  }
  __syncthreads();
  const int t = threadIdx.x;
  float sum = 0.f;
  if (t < kBiasCols)
    for (int w = 0; w < warps; ++w) sum += part[w][t];
  if (ranks > 1) {
    __syncthreads();
    if (t < kBiasCols) part[0][t] = sum;
    cluster_sync();
    if (rank == 0 && t < kBiasCols)
      for (int r = 1; r < ranks; ++r) sum += ld_cluster_f32(mapa(smem_u32(&part[0][t]), r));
    cluster_sync();                                  // the others' shared memory has been read
  }
  const int n = at % blocks * kBiasCols + t;
  if (rank == 0 && t < kBiasCols && n < l.T) {
    float* o = out + (int64_t)g * l.T + n;
    *o = add ? *o + sum : sum;
  }
  if (l.beside) ops_end_beside();
}

moe_status bias_grad(const Args* a, const void* grad, int64_t grad_stride, bool beside, int sms, void* s) {
  LinearParams l = {};
  l.beside = beside;
  l.T = a->fan_out;
  l.F = a->rows;
  l.G = std::max(1, a->groups);
  l.offsets = a->d_offsets;
  const int64_t blocks = (int64_t)((l.T + kBiasCols - 1) / kBiasCols) * l.G;
  // a CTA for some 64 rows of an average group, as long as there are few
  int ranks = 1;
  while (ranks < kBiasRanks && (int64_t)a->rows / l.G > 64 * ranks && blocks * ranks < 4 * sms) ranks *= 2;
  return launch_op(grad_bias_kernel, dim3((unsigned)(blocks * ranks)), kBiasThreads, 0, ranks, s, static_cast<const __nv_bfloat16*>(grad), grad_stride, l,
                   a->d_grad_bias, a->accumulate);
}

// Rows that do not start on 16-byte boundaries, which the copies into shared memory need: put on such boundaries first.
__global__ void __launch_bounds__(256)
    align_rows_kernel(const __nv_bfloat16* __restrict__ in, int64_t ld, __nv_bfloat16* __restrict__ out, int64_t ldo, int T, int N) {
  ops_begin();
  const int c = blockIdx.x * 256 + threadIdx.x;
  constexpr int kRows = 4;
  const int64_t row = ((int64_t)blockIdx.z * 65535 + blockIdx.y) * kRows;
  if (c >= N) return;
  __nv_bfloat16 v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (row + i < T) v[i] = in[(row + i) * ld + c];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (row + i < T) out[(row + i) * ldo + c] = v[i];
}

int64_t aligned_stride(int32_t fan_out) { return ((int64_t)fan_out + 7) / 8 * 8; }

// ------------------------------------------------------------------ the epilogue's gradient

// act'(z) and act(z).  z is taken as +-128 beyond: every slope there is 0 or 1 in fp32, and infinities do not meet zeros.
template <typename T>
__device__ __forceinline__ void act_and_slope(int act, float z, float& y, float& slope) {
  const float c = z > 128.f ? 128.f : z < -128.f ? -128.f : z;              // NaN stays
  if (act == MOE_ACT_SILU) {
    // s = 1 / (1 + e^-z) and 1 - s, each without cancellation: slope = s (1 + z (1 - s))
    const float e = sizeof(T) == 4 ? expf(-fabsf(c)) : __expf(-fabsf(c)), r = __fdividef(1.0f, 1.0f + e);
    const float s = c < 0.f ? e * r : r, o = c < 0.f ? r : e * r;
    y = silu<T>(z);
    slope = s * fmaf(c, o, 1.0f);
  } else if (act == MOE_ACT_GELU) {
    float density;                                   // sqrt(2 pi) times the normal density
    const float cdf = normal_cdf<T>(c, density);
    y = z * cdf;
    slope = fmaf(c * 0.398942280f, density, cdf);
  } else if (act == MOE_ACT_RELU) {
    y = z < 0.f ? 0.f : z;
    slope = z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
  } else {
    y = z;
    slope = 1.f;
  }
}

// a b slope, the larger factor first: a b may lie outside fp32 where the result, of a slope of 0 say, does not.  The sign goes with the
// larger one; NaN stays.
__device__ __forceinline__ float triple(float a, float b, float slope) {
  float large, small;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(large) : "f"(a), "f"(b));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(small) : "f"(fabsf(a)), "f"(fabsf(b)));
  return large * slope * small;
}

template <typename T> struct ActParams {
  Rows<const T> grad, z, mul;
  Rows<T> grad_z, grad_mul;
  int64_t width;
  int chunks, act;
};

// Bound by memory: three reads and two writes (8192 x 2880 bf16 36.1 us, 96% of the copy rate).  A thread asks for all that its kU
// units need before it uses the first.  The outputs may be the inputs: every element is read by the thread that writes it, before.
template <typename T, int V, bool MUL>
__global__ void __launch_bounds__(256) act_mul_backward_kernel(const ActParams<T> p) {
  using RV = RowVec<T, V>;
  constexpr int kU = 2;
  ops_begin();
  const int64_t row = blockIdx.x / p.chunks;
  const int64_t c0 = ((int64_t)(blockIdx.x % p.chunks) * kU * 256 + threadIdx.x) * V;
  typename RV::Raw g[kU], z[kU], m[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t c = c0 + u * 256 * V;
    if (c >= p.width) continue;
    g[u] = RV::load_rw(p.grad.at(row) + c);
    z[u] = RV::load_rw(p.z.at(row) + c);
    if (MUL) m[u] = RV::load_rw(p.mul.at(row) + c);
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t c = c0 + u * 256 * V;
    if (c >= p.width) continue;
    float gv[V], zv[V], mv[V], oz[V], om[V];
    RV::unpack(g[u], gv);
    RV::unpack(z[u], zv);
    if (MUL) RV::unpack(m[u], mv);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float y, slope;
      act_and_slope<T>(p.act, zv[i], y, slope);
      oz[i] = MUL ? triple(gv[i], mv[i], slope) : gv[i] * slope;
      om[i] = gv[i] * y;
    }
    RV::store(p.grad_z.at(row) + c, RV::pack(oz));
    if (MUL) RV::store(p.grad_mul.at(row) + c, RV::pack(om));
  }
}

template <typename T, int V>
moe_status launch_act(ActParams<T> p, int64_t rows, void* s) {
  const int64_t per = 2 * 256 * V, chunks = (p.width + per - 1) / per;
  if (chunks > INT32_MAX || rows * chunks > INT32_MAX) return MOE_ERR_INVALID;
  p.chunks = (int)chunks;
  return launch_op(p.mul.p ? act_mul_backward_kernel<T, V, true> : act_mul_backward_kernel<T, V, false>, dim3((unsigned)(rows * chunks)), 256, 0, 1, s, p);
}

template <typename T>
moe_status act_backward(int32_t act, const void* grad, int64_t ldg, const void* z, int64_t ldz, const void* mul, int64_t ldm, int64_t rows, int64_t width,
                        void* gz, int64_t ldgz, void* gm, int64_t ldgm, void* s) {
  ActParams<T> p{{static_cast<const T*>(grad), ldg}, {static_cast<const T*>(z), ldz}, {static_cast<const T*>(mul), ldm},
                 {static_cast<T*>(gz), ldgz}, {static_cast<T*>(gm), ldgm}, width, 0, act};
  if (rows == 1 || (ldg == width && ldz == width && ldgz == width && (!mul || (ldm == width && ldgm == width)))) {
    p.width = rows * width;                          // whole matrices: one long row
    rows = 1;
  }
  constexpr int size = sizeof(T);
  const auto units = [&](const void* q, int64_t ld) { return !q || (aligned16(q) && (rows == 1 || ld * size % 16 == 0)); };
  const bool wide = p.width * size % 16 == 0 && units(grad, ldg) && units(z, ldz) && units(mul, ldm) && units(gz, ldgz) && units(gm, ldgm);
  return wide ? launch_act<T, Vec<T>::N>(p, rows, s) : launch_act<T, 1>(p, rows, s);
}

}  // namespace

unsigned int* ops_error_backward() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_ops_error) == cudaSuccess ? static_cast<unsigned int*>(p) : nullptr;
}

}  // namespace moe

extern "C" int64_t moe_async_linear_backward_workspace(const moe_async_linear_backward_args* a) {
  using namespace moe;
  if (!a || a->rows < 1 || a->fan_out < 1 || rows16(a->d_grad, a->grad_stride, 2)) return 0;
  return a->rows * aligned_stride(a->fan_out) * 2;
}

extern "C" moe_status moe_async_linear_backward(const moe_async_linear_backward_args* a, void* stream) {
  using namespace moe;
  if (!a) return MOE_ERR_INVALID;
  if (a->rows < 0 || a->rows > kMaxRows || a->fan_in < 1 || a->fan_in > INT32_MAX - 1024 || a->fan_out < 1 ||
      a->fan_out > INT32_MAX - 1024 || a->groups < 0 || a->groups > kMaxExperts || (a->groups > 0) != (a->d_offsets != nullptr) ||
      (a->x_dtype != MOE_F32 && a->x_dtype != MOE_BF16) || (a->w_dtype != MOE_F32 && a->w_dtype != MOE_BF16))
    return MOE_ERR_INVALID;
  const bool gx = a->d_grad_x != nullptr, gw = a->d_grad_w != nullptr, gb = a->d_grad_bias != nullptr;
  const int64_t G = std::max(1, a->groups);
  if ((gx && (!a->d_w || a->w_stride < a->fan_in || a->grad_x_stride < a->fan_in)) || (a->d_residual && (!gx || a->residual_stride < a->fan_in)) ||
      (gw && a->grad_w_stride < a->fan_in))
    return MOE_ERR_INVALID;
  // tiles are counted in 32 bits
  if (((int64_t)a->fan_out / 64 + 1) * ((int64_t)a->fan_in / 128 + 1) * G * 8 > INT32_MAX ||
      ((int64_t)a->rows / 16 + G + 1) * ((int64_t)a->fan_in / 128 + 1) * 8 > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->rows == 0) {                                // sums of nothing
    if (a->accumulate) return MOE_OK;
    const size_t size = dtype_size(a->w_dtype);
    if (gw && cudaMemset2DAsync(a->d_grad_w, a->grad_w_stride * size, 0, a->fan_in * size, G * a->fan_out, s) != cudaSuccess) return MOE_ERR_CUDA;
    if (gb && cudaMemsetAsync(a->d_grad_bias, 0, G * a->fan_out * sizeof(float), s) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!a->d_grad || a->grad_stride < a->fan_out || (gw && (!a->d_x || a->x_stride < a->fan_in))) return MOE_ERR_INVALID;
  if (a->fan_in % 8 || (gx && !rows16(a->d_w, a->w_stride, 2)) || (gw && !rows16(a->d_x, a->x_stride, 2))) return MOE_ERR_UNSUPPORTED;
  const int64_t need = moe_async_linear_backward_workspace(a);
  if (need > 0) {
    if (!a->d_workspace || !aligned16(a->d_workspace)) return MOE_ERR_INVALID;
    if (a->workspace_bytes < need) return MOE_ERR_CAPACITY;
  }
  // the three run beside each other: what one writes, the others must not read
  const void* const in[] = {a->d_grad, gw ? a->d_x : nullptr, gx ? a->d_w : nullptr, a->d_workspace};
  for (const void* i : in)
    if (i && (i == a->d_grad_x || i == a->d_grad_w || i == a->d_grad_bias)) return MOE_ERR_INVALID;
  if ((gw && (a->d_grad_w == a->d_grad_x || a->d_grad_w == a->d_residual)) || (gb && (a->d_grad_bias == a->d_grad_x || a->d_grad_bias == a->d_grad_w)))
    return MOE_ERR_INVALID;
  const int sms = sm_count();
  if (sms < 2) return MOE_ERR_CUDA;
  const void* grad = a->d_grad;
  int64_t ld = a->grad_stride;
  moe_status r = MOE_OK;
  if (need > 0) {
    ld = aligned_stride(a->fan_out);
    const int64_t y = ((int64_t)a->rows + 3) / 4;
    const dim3 grid((unsigned)((a->fan_out + 255) / 256), (unsigned)std::min<int64_t>(y, 65535), (unsigned)((y + 65534) / 65535));
    r = launch_op(align_rows_kernel, grid, 256, 0, 1, s, static_cast<const __nv_bfloat16*>(grad), a->grad_stride,
                  static_cast<__nv_bfloat16*>(a->d_workspace), ld, a->rows, a->fan_out);
    grad = a->d_workspace;
  }
  if (r == MOE_OK && gx) r = a->x_dtype == MOE_F32 ? rows_grad<float>(a, grad, ld, sms, s) : rows_grad<__nv_bfloat16>(a, grad, ld, sms, s);
  // The three need nothing of each other: the first waits for what came before, the others run beside it as it leaves room.
  if (r == MOE_OK && gw)
    r = a->w_dtype == MOE_F32 ? weight_grad<float>(a, grad, ld, gx, sms, s) : weight_grad<__nv_bfloat16>(a, grad, ld, gx, sms, s);
  if (r == MOE_OK && gb) r = bias_grad(a, grad, ld, gx || gw, sms, s);
  return r;
}

extern "C" moe_status moe_async_act_mul_backward(int32_t dtype, int32_t act, const void* d_grad, int64_t grad_stride, const void* d_z, int64_t z_stride,
                                                 const void* d_mul, int64_t mul_stride, int32_t T, int32_t H, void* d_grad_z, int64_t grad_z_stride,
                                                 void* d_grad_mul, int64_t grad_mul_stride, void* stream) {
  using namespace moe;
  if (T < 0 || H < 1 || H > kMaxWidth || act < MOE_ACT_NONE || act > MOE_ACT_RELU || (dtype != MOE_F32 && dtype != MOE_BF16) ||
      (d_mul != nullptr) != (d_grad_mul != nullptr))
    return MOE_ERR_INVALID;
  if (T == 0) return MOE_OK;
  if (!d_grad || !d_z || !d_grad_z || grad_stride < H || z_stride < H || grad_z_stride < H || (d_mul && (mul_stride < H || grad_mul_stride < H)) ||
      d_grad_z == d_grad_mul)
    return MOE_ERR_INVALID;
  return dtype == MOE_F32 ? act_backward<float>(act, d_grad, grad_stride, d_z, z_stride, d_mul, mul_stride, T, H, d_grad_z, grad_z_stride, d_grad_mul,
                                                grad_mul_stride, stream)
                          : act_backward<__nv_bfloat16>(act, d_grad, grad_stride, d_z, z_stride, d_mul, mul_stride, T, H, d_grad_z, grad_z_stride,
                                                        d_grad_mul, grad_mul_stride, stream);
}
