// Root-mean-square norm with the residual's addition, its 8-bit form and its gradient.
//
//   h = x + residual, rounded to the rows' type (the residual stream the next layer adds to)
//   y = h * r * gain,  r = 1 / sqrt(mean(h^2) + eps), taken over the rounded h
//   e4m3: scale = max(max|y| / 448, 2^-126) per row, q = y / scale
//   backward, u = grad_y * gain, n = h * r:
//     grad_x = r (u - n mean(u n)) + grad_h,   grad_gain = sum over rows of grad_y * n
//
// One pass over the row: max|y| = r max|h gain|, so the sum of squares and the maximum come from
// the same reduction.  Sums are fp32 in a fixed order (no atomics).
#include <cuda_fp8.h>
#include <algorithm>
#include "moe_ops.cuh"

namespace moe {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;         // 2^-126

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct SumMax {
  float s, m;
};

// Sum and NaN-keeping maximum over a block of up to 32 warps, the same value in every thread.
__device__ __forceinline__ SumMax block_sum_max(SumMax v, SumMax* part) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    v.s += __shfl_xor_sync(0xffffffffu, v.s, off);
    v.m = max_nan(v.m, __shfl_xor_sync(0xffffffffu, v.m, off));
  }
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  __syncthreads();                                   // `part` may still be read from the row before
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  SumMax a = part[0];
  for (int i = 1; i < warps; ++i) {
    a.s += part[i].s;
    a.m = max_nan(a.m, part[i].m);
  }
  return a;
}

template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t* q, const float (&v)[V]) {
  if constexpr (V == 1) {
    *q = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | hi << 16;
    }
    if constexpr (V == 8)
      *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(q) = w[0];
  }
}

// One block per row.  The row stays in registers up to NV units a thread; what lies behind them
// is read again.
template <typename T, int V, int NV, bool Q>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(Rows<const T> x, Rows<const T> res,
                                                            const float* __restrict__ gain, float eps, int H,
                                                            Rows<T> hout, Rows<T> y, Rows<uint8_t> q,
                                                            float* __restrict__ scale) {
  using RV = RowVec<T, V>;
  __shared__ SumMax part[32];
  ops_begin();
  const long long t = blockIdx.x;
  const int step = blockDim.x * V, c0 = threadIdx.x * V;
  typename RV::Raw keep[NV];
  SumMax a{0.f, 0.f};
  auto sum = [&](int c) {
    typename RV::Raw r = RV::load_rw(x.at(t) + c);
    if (res.p) {
      float v[V], o[V];
      RV::unpack(r, v);
      RV::unpack(RV::load_rw(res.at(t) + c), o);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += o[i];
      r = RV::pack(v);
    }
    return r;
  };
  auto take = [&](int c) {
    const typename RV::Raw r = sum(c);
    if (hout.p) RV::store(hout.at(t) + c, r);
    float v[V];
    RV::unpack(r, v);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      a.s = fmaf(v[i], v[i], a.s);
      if (Q) a.m = max_nan(a.m, fabsf(gain ? v[i] * __ldg(gain + c + i) : v[i]));
    }
    return r;
  };
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (c0 + j * step < H) keep[j] = take(c0 + j * step);
  for (int c = c0 + NV * step; c < H; c += step) take(c);
  a = block_sum_max(a, part);
  const float r = 1.0f / sqrtf(a.s / (float)H + eps);
  const float sc = max_nan(r * a.m * (1.0f / kE4m3Max), kMinScale), inv = 1.0f / sc;
  if (Q && threadIdx.x == 0) scale[t] = sc;
  auto give = [&](int c, const typename RV::Raw& raw) {
    float v[V];
    RV::unpack(raw, v);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = (gain ? v[i] * __ldg(gain + c + i) : v[i]) * r;
      if (Q) v[i] *= inv;
    }
    if constexpr (Q)
      store_e4m3<V>(q.at(t) + c, v);
    else
      RV::store(y.at(t) + c, RV::pack(v));
  };
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (c0 + j * step < H) give(c0 + j * step, keep[j]);
  // h may have taken the place of x or of the residual: what this thread wrote is read
  for (int c = c0 + NV * step; c < H; c += step) give(c, hout.p ? RV::load_rw(hout.at(t) + c) : sum(c));
}

// Rows blockIdx.x, + gridDim.x, ...; every block leaves the sum of grad_y * n over its rows in
// its row of `partial` [gridDim.x, H].
template <typename T, int V>
__global__ void __launch_bounds__(256) rms_norm_backward_kernel(Rows<const T> gy, Rows<const T> h,
                                                                const float* __restrict__ gain, float eps, int T_,
                                                                int H, Rows<const T> gh, Rows<T> gx,
                                                                float* __restrict__ partial) {
  using RV = RowVec<T, V>;
  __shared__ SumMax part[32];
  ops_begin();
  float* mine = partial ? partial + (size_t)blockIdx.x * H : nullptr;
  bool first = true;
  for (long long t = blockIdx.x; t < T_; t += gridDim.x) {
    SumMax a{0.f, 0.f}, b{0.f, 0.f};
    for (int c = threadIdx.x * V; c < H; c += blockDim.x * V) {
      float g[V], v[V];
      RV::unpack(RV::load(gy.at(t) + c), g);
      RV::unpack(RV::load(h.at(t) + c), v);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a.s = fmaf(v[i], v[i], a.s);
        b.s = fmaf(gain ? g[i] * __ldg(gain + c + i) : g[i], v[i], b.s);
      }
    }
    a = block_sum_max(a, part);
    b = block_sum_max(b, part);
    const float r = 1.0f / sqrtf(a.s / (float)H + eps);
    const float m = r * (b.s / (float)H);            // mean(u n)
    for (int c = threadIdx.x * V; c < H; c += blockDim.x * V) {
      float g[V], v[V], o[V], e[V];
      RV::unpack(RV::load(gy.at(t) + c), g);
      RV::unpack(RV::load(h.at(t) + c), v);
      if (gh.p) RV::unpack(RV::load_rw(gh.at(t) + c), e);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float n = v[i] * r, u = gain ? g[i] * __ldg(gain + c + i) : g[i];
        o[i] = r * (u - n * m);
        if (gh.p) o[i] += e[i];
        if (mine) mine[c + i] = first ? g[i] * n : mine[c + i] + g[i] * n;
      }
      RV::store(gx.at(t) + c, RV::pack(o));
    }
    first = false;
  }
}

__global__ void __launch_bounds__(256) sum_partials_kernel(const float* __restrict__ partial, int G, int H,
                                                           float* __restrict__ out) {
  ops_begin();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= H) return;
  float a = 0.f;
  for (int g = 0; g < G; ++g) a += partial[(size_t)g * H + c];
  out[c] = a;
}

template <typename T, int V, bool Q>
moe_status norm_launch(const Rows<const T>& x, const Rows<const T>& res, const float* gain, float eps, int T_, int H,
                       const Rows<T>& h, const Rows<T>& y, const Rows<uint8_t>& q, float* scale, void* s) {
  const int units = (H + V - 1) / V;
  const int threads = std::min(1024, std::max(32, (units + 3) / 4 + 31 & ~31));
  return launch_op(add_rms_norm_kernel<T, V, 4, Q>, dim3(T_), threads, 0, 1, s, x, res, gain, eps, H, h, y, q, scale);
}

template <typename T>
moe_status norm_dispatch(const void* x, int64_t ldx, const void* res, int64_t ldr, const float* gain, float eps, int T_,
                         int H, void* h, int64_t ldh, void* y, int64_t ldy, float* scale, void* s) {
  constexpr int N = Vec<T>::N;
  const Rows<const T> xr{static_cast<const T*>(x), ldx}, rr{static_cast<const T*>(res), ldr};
  const Rows<T> hr{static_cast<T*>(h), ldh};
  const Rows<T> yr{scale ? nullptr : static_cast<T*>(y), ldy};
  const Rows<uint8_t> qr{scale ? static_cast<uint8_t*>(y) : nullptr, ldy};
  const bool wide = H % N == 0 && rows16(x, ldx, sizeof(T)) && rows16(res, ldr, sizeof(T)) && rows16(h, ldh, sizeof(T));
  if (scale) {
    if (wide && reinterpret_cast<uintptr_t>(y) % N == 0 && ldy % N == 0)
      return norm_launch<T, N, true>(xr, rr, gain, eps, T_, H, hr, yr, qr, scale, s);
    return norm_launch<T, 1, true>(xr, rr, gain, eps, T_, H, hr, yr, qr, scale, s);
  }
  if (wide && rows16(y, ldy, sizeof(T)))
    return norm_launch<T, N, false>(xr, rr, gain, eps, T_, H, hr, yr, qr, scale, s);
  return norm_launch<T, 1, false>(xr, rr, gain, eps, T_, H, hr, yr, qr, scale, s);
}

// Blocks of the backward pass: the rows of `partial`.
constexpr int kNormBwdBlocks = 304;
int norm_bwd_blocks(int T_) { return std::min(T_, kNormBwdBlocks); }

template <typename T>
moe_status norm_backward_dispatch(const void* gy, int64_t ldgy, const void* h, int64_t ldh, const float* gain, float eps,
                                  int T_, int H, const void* gh, int64_t ldgh, void* gx, int64_t ldgx, float* ggain,
                                  float* ws, void* s) {
  constexpr int N = Vec<T>::N;
  const Rows<const T> a{static_cast<const T*>(gy), ldgy}, b{static_cast<const T*>(h), ldh},
      c{static_cast<const T*>(gh), ldgh};
  const Rows<T> o{static_cast<T*>(gx), ldgx};
  const int G = norm_bwd_blocks(T_);
  float* partial = ggain ? ws : nullptr;
  const bool wide = H % N == 0 && rows16(gy, ldgy, sizeof(T)) && rows16(h, ldh, sizeof(T)) &&
                    rows16(gh, ldgh, sizeof(T)) && rows16(gx, ldgx, sizeof(T));
  moe_status st = wide ? launch_op(rms_norm_backward_kernel<T, N>, dim3(G), 256, 0, 1, s, a, b, gain, eps, T_, H, c, o,
                                   partial)
                       : launch_op(rms_norm_backward_kernel<T, 1>, dim3(G), 256, 0, 1, s, a, b, gain, eps, T_, H, c, o,
                                   partial);
  if (st != MOE_OK || !ggain) return st;
  return launch_op(sum_partials_kernel, dim3((H + 255) / 256), 256, 0, 1, s, (const float*)ws, G, H, ggain);
}

}  // namespace
}  // namespace moe

extern "C" {
using namespace moe;

moe_status moe_async_add_rms_norm(int32_t dtype, const void* d_x, int64_t x_stride, const void* d_residual,
                                  int64_t residual_stride, const float* d_gain, float eps, int32_t T, int32_t H,
                                  void* d_h, int64_t h_stride, void* d_y, int64_t y_stride, float* d_scale,
                                  void* stream) {
  if ((dtype != MOE_F32 && dtype != MOE_BF16) || T < 0 || H < 1 || !(eps >= 0.f)) return MOE_ERR_INVALID;
  if (T == 0) return MOE_OK;
  if (!d_x || !d_y || x_stride < H || y_stride < H || (d_residual && residual_stride < H) ||
      (d_h && (!d_residual || h_stride < H)))
    return MOE_ERR_INVALID;
  return dtype == MOE_BF16
             ? norm_dispatch<__nv_bfloat16>(d_x, x_stride, d_residual, residual_stride, d_gain, eps, T, H, d_h, h_stride,
                                            d_y, y_stride, d_scale, stream)
             : norm_dispatch<float>(d_x, x_stride, d_residual, residual_stride, d_gain, eps, T, H, d_h, h_stride, d_y,
                                    y_stride, d_scale, stream);
}

int64_t moe_async_add_rms_norm_backward_workspace(int32_t T, int32_t H) {
  return T < 1 || H < 1 ? 0 : (int64_t)norm_bwd_blocks(T) * H * (int64_t)sizeof(float);
}

moe_status moe_async_add_rms_norm_backward(int32_t dtype, const void* d_grad, int64_t grad_stride, const void* d_h,
                                           int64_t h_stride, const float* d_gain, float eps, int32_t T, int32_t H,
                                           const void* d_grad_h, int64_t grad_h_stride, void* d_grad_x,
                                           int64_t grad_x_stride, float* d_grad_gain, void* d_workspace,
                                           int64_t workspace_bytes, void* stream) {
  if ((dtype != MOE_F32 && dtype != MOE_BF16) || T < 0 || H < 1 || !(eps >= 0.f)) return MOE_ERR_INVALID;
  if (T == 0) {
    if (!d_grad_gain) return MOE_OK;
    return cudaMemsetAsync(d_grad_gain, 0, (size_t)H * sizeof(float), static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  }
  if (!d_grad || !d_h || !d_grad_x || grad_stride < H || h_stride < H || grad_x_stride < H ||
      (d_grad_h && grad_h_stride < H))
    return MOE_ERR_INVALID;
  if (d_grad_gain) {
    if (!d_workspace || reinterpret_cast<uintptr_t>(d_workspace) % 16) return MOE_ERR_INVALID;
    if (workspace_bytes < moe_async_add_rms_norm_backward_workspace(T, H)) return MOE_ERR_CAPACITY;
  }
  float* ws = static_cast<float*>(d_workspace);
  return dtype == MOE_BF16
             ? norm_backward_dispatch<__nv_bfloat16>(d_grad, grad_stride, d_h, h_stride, d_gain, eps, T, H, d_grad_h,
                                                     grad_h_stride, d_grad_x, grad_x_stride, d_grad_gain, ws, stream)
             : norm_backward_dispatch<float>(d_grad, grad_stride, d_h, h_stride, d_gain, eps, T, H, d_grad_h,
                                             grad_h_stride, d_grad_x, grad_x_stride, d_grad_gain, ws, stream);
}

}  // extern "C"
