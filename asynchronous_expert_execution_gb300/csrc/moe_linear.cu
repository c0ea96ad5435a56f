// Matrix product with its epilogue, dense or per expert on sorted rows:
//
//   y[t, n] = act(sx[t] sw[n] sum_k x[t, k] w[n, k] + bias[n]) * mul[t, n] + residual[t, n]
//
// x [T, F] and w [N, F] (or [G, N, F]: rows offsets[g] .. offsets[g + 1] of x meet w[g]) in bf16 or
// e4m3, products summed in fp32, y in bf16 or fp32, rounded once.
//
// Three kernels, chosen by expected time (linear_launch, linear_plan): pair and split (moe_linear.cuh), with both
// operands K-major as they lie in memory, and
//   few    up to 16 tokens: weights straight into the registers of warp-wide matrix instructions.  Only
//          the weights' bytes count there; barriers, TMEM and the exchange cost more than they bring
//          (4 tokens on 2880 x 2880: 5.8 us against 7.0).
#include "moe_linear.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------ few tokens

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
  if (bn > 64 || (tiles * splits <= split_capacity<kForward>(splits, sms) && l.nk > p.stages * splits)) p.stages = split_stages(bn, true);
  const int stage = kABlock + bn * kBKBytes, rest = (int)sizeof(SplitTail) + 1024;
  const int smem = p.stages * stage + rest;
  if (!encode(&p.w, a->d_w, size, l.F, l.N, a->w_stride, l.G, kBM) ||
      !encode(&p.x, a->d_x, size, l.F, l.T, a->x_stride, 0, bn))
    return MOE_ERR_CUDA;
  if (cudaFuncSetAttribute(linear_split_kernel<E4M3, TO>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmem) != cudaSuccess)
    return MOE_ERR_CUDA;
  return launch_op(linear_split_kernel<E4M3, TO>, dim3((unsigned)(tiles * splits)), kThreads, smem, splits, s, p);
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

namespace moe {
// every set of product kernels has an error word of its own
unsigned int* ops_error_backward();
unsigned int* ops_error_blocks();
}

namespace {
constexpr int kWords = 3;

// The words of the current device; false: one is not to be had.
bool error_words(unsigned int* (&words)[kWords]) {
  void* mine = nullptr;
  if (cudaGetSymbolAddress(&mine, moe::g_ops_error) != cudaSuccess) return false;
  words[0] = static_cast<unsigned int*>(mine);
  words[1] = moe::ops_error_backward();
  words[2] = moe::ops_error_blocks();
  return words[1] && words[2];
}
}  // namespace

extern "C" moe_status moe_async_ops_status(void* stream) {
  unsigned int* words[kWords];
  if (!error_words(words)) return MOE_ERR_CUDA;
  unsigned int e[kWords] = {};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int i = 0; i < kWords; ++i)
    if (cudaMemcpyAsync(&e[i], words[i], sizeof(e[i]), cudaMemcpyDeviceToHost, s) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return MOE_ERR_CUDA;
  unsigned int found = 0;
  for (int i = 0; i < kWords; ++i) {
    if (e[i] == 0) continue;
    found = e[i];                                    // reported: the calls after this one start clear
    if (cudaMemsetAsync(words[i], 0, sizeof(e[i]), s) != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (found != 0 && cudaStreamSynchronize(s) != cudaSuccess) return MOE_ERR_CUDA;
  return static_cast<moe_status>(found);
}

extern "C" moe_status moe_async_debug_latch_ops_word(int32_t word, void* stream) {
#ifdef MOE_DEBUG_BOUNDS
  unsigned int* words[kWords];
  if (word < 0 || word >= kWords) return MOE_ERR_INVALID;
  if (!error_words(words)) return MOE_ERR_CUDA;
  const unsigned int e = MOE_ERR_TIMEOUT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cudaMemcpyAsync(words[word], &e, sizeof(e), cudaMemcpyHostToDevice, s) == cudaSuccess && cudaStreamSynchronize(s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
#else
  (void)word;
  (void)stream;
  return MOE_ERR_UNSUPPORTED;
#endif
}

extern "C" moe_status moe_async_debug_latch_ops_error(void* stream) { return moe_async_debug_latch_ops_word(0, stream); }
