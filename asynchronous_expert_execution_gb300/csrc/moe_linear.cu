// Matrix product with its epilogue, dense or per expert on sorted rows:
//
//   y[t, n] = act(sx[t] sw[n] sum_k x[t, k] w[n, k] + bias[n]) * mul[t, n] + residual[t, n]
//
// x [T, F] and w [N, F] (or [G, N, F]: rows offsets[g] .. offsets[g + 1] of x meet w[g]) in bf16 or
// e4m3, products summed in fp32, y in bf16 or fp32, rounded once.
#include <cuda_fp8.h>
#include <algorithm>
#include "moe_ops.cuh"

namespace moe {
namespace {

struct LinearParams {
  const void* x;
  const void* w;
  const float* bias;
  const float* sx;
  const float* sw;
  const void* mul;
  const void* res;
  void* y;
  const int32_t* offsets;
  int64_t ldx, ldw, ldmul, ldres, ldy;
  int T, N, F, G, act;
};

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case MOE_ACT_SILU: return v / (1.0f + expf(-v));
    case MOE_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678f));
    case MOE_ACT_RELU: return v < 0.f ? 0.f : v;     // NaN stays
    default: return v;
  }
}

__device__ __forceinline__ float operand(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ float operand(const __nv_fp8_e4m3* p, int64_t i) { return float(p[i]); }

constexpr int kTile = 32;

// 32 x 32 outputs a block, one a thread, operands staged in shared memory as fp32.
template <typename TI, typename TO>
__global__ void __launch_bounds__(1024) linear_kernel(LinearParams p) {
  __shared__ float xs[kTile][kTile + 1], ws[kTile][kTile + 1];
  ops_begin();
  int g = 0, r0 = blockIdx.y * kTile, r1 = p.T;
  if (p.offsets) {
    int tile = blockIdx.y;
    for (; g < p.G; ++g) {
      const int a = min(p.T, max(0, p.offsets[g])), b = min(p.T, max(a, p.offsets[g + 1]));
      const int n = (b - a + kTile - 1) / kTile;
      if (tile < n) {
        r0 = a + tile * kTile;
        r1 = b;
        break;
      }
      tile -= n;
    }
    if (g == p.G) return;
  }
  const TI* x = static_cast<const TI*>(p.x);
  const TI* w = static_cast<const TI*>(p.w) + (size_t)g * p.N * p.ldw;
  const int n0 = blockIdx.x * kTile, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  float acc = 0.f;
  for (int k0 = 0; k0 < p.F; k0 += kTile) {
    const int k = k0 + tx;
    xs[ty][tx] = r0 + ty < r1 && k < p.F ? operand(x, (r0 + ty) * p.ldx + k) : 0.f;
    ws[ty][tx] = n0 + ty < p.N && k < p.F ? operand(w, (int64_t)(n0 + ty) * p.ldw + k) : 0.f;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kTile; ++j) acc = fmaf(xs[ty][j], ws[tx][j], acc);
    __syncthreads();
  }
  const long long r = r0 + ty;
  const int n = n0 + tx;
  if (r >= r1 || n >= p.N) return;
  if (p.sx) acc = acc * p.sx[r] * p.sw[(size_t)g * p.N + n];
  if (p.bias) acc += p.bias[(size_t)g * p.N + n];
  acc = activate(acc, p.act);
  if (p.mul) acc *= to_f(static_cast<const TO*>(p.mul)[r * p.ldmul + n]);
  if (p.res) acc += to_f(static_cast<const TO*>(p.res)[r * p.ldres + n]);
  static_cast<TO*>(p.y)[r * p.ldy + n] = from_f<TO>(acc);
}

template <typename TI>
moe_status linear_launch(const LinearParams& p, int32_t out_dtype, void* s) {
  const int tiles = p.T / kTile + (p.offsets ? p.G : 1);         // at least one per row tile of every group
  const dim3 grid((p.N + kTile - 1) / kTile, tiles);
  return out_dtype == MOE_BF16 ? launch_op(linear_kernel<TI, __nv_bfloat16>, grid, 1024, 0, 1, s, p)
                               : launch_op(linear_kernel<TI, float>, grid, 1024, 0, 1, s, p);
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_async_linear(const moe_async_linear_args* a, void* stream) {
  using namespace moe;
  if (!a) return MOE_ERR_INVALID;
  if (a->rows < 0 || a->fan_in < 1 || a->fan_out < 1 || a->groups < 0 || a->groups > kMaxExperts ||
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
  if (a->fan_in * size % 16 || !rows16(a->d_x, a->x_stride, size) || !rows16(a->d_w, a->w_stride, size))
    return MOE_ERR_UNSUPPORTED;
  LinearParams p{a->d_x,      a->d_w,      a->d_bias,   a->d_x_scale,  a->d_w_scale,       a->d_mul,    a->d_residual,
                 a->d_y,      a->d_offsets, a->x_stride, a->w_stride,  a->mul_stride,      a->residual_stride,
                 a->y_stride, a->rows,     a->fan_out,  a->fan_in,     std::max(1, a->groups), a->act};
  return e4m3 ? linear_launch<__nv_fp8_e4m3>(p, a->out_dtype, stream)
              : linear_launch<__nv_bfloat16>(p, a->out_dtype, stream);
}
