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

// Sum of a and, as MAX says, NaN-keeping maximum or sum of b, over the G threads of a row (32, or
// the whole block), the same values in every thread.
template <int G, bool MAX>
__device__ __forceinline__ void row_reduce(float& a, float& b, float2* part) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, off);
    const float o = __shfl_xor_sync(0xffffffffu, b, off);
    b = MAX ? max_nan(b, o) : b + o;
  }
  if (G == 32) return;
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();                                   // `part` may still be read for the row before
  if (lane == 0) part[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < warps ? part[lane] : make_float2(0.f, 0.f);
  a = v.x;
  b = v.y;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, off);
    const float o = __shfl_xor_sync(0xffffffffu, b, off);
    b = MAX ? max_nan(b, o) : b + o;
  }
}

// The gain of a unit of V columns (all ones without one); wide units start on 16 bytes.
template <int V>
__device__ __forceinline__ void load_gain(const float* gain, int c, float (&g)[V]) {
  if constexpr (V == 1) {
    g[0] = gain ? __ldg(gain + c) : 1.f;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 v = gain ? __ldg(reinterpret_cast<const float4*>(gain + c + i)) : make_float4(1.f, 1.f, 1.f, 1.f);
      g[i] = v.x, g[i + 1] = v.y, g[i + 2] = v.z, g[i + 3] = v.w;
    }
  }
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

// Bound by memory: one read of x and the residual, one write of h and y.  A row belongs to G
// threads -- a warp (four rows a block) where it fits one, else a block -- and stays in their
// registers, NV units a thread, all loads issued before the first is used; what lies behind
// them is read again.
template <typename T, int V, int NV, int G, bool Q>
__global__ void __launch_bounds__(G == 32 ? 128 : V == 1 ? 1024 : 512, 1)
    add_rms_norm_kernel(Rows<const T> x, Rows<const T> res, const float* __restrict__ gain, float eps, int T_, int H,
                        Rows<T> hout, Rows<T> y, Rows<uint8_t> q, float* __restrict__ scale) {
  using RV = RowVec<T, V>;
  __shared__ float2 part[32];
  ops_begin();
  const int threads = G == 32 ? 32 : blockDim.x, tid = G == 32 ? threadIdx.x & 31 : threadIdx.x;
  const long long t = G == 32 ? (long long)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= T_) return;                               // whole warps
  const int step = threads * V, c0 = tid * V;
  typename RV::Raw keep[NV], add[NV];
  float ss = 0.f, mx = 0.f;
  auto sum = [&](const typename RV::Raw& a, const typename RV::Raw& b) {
    float v[V], o[V];
    RV::unpack(a, v);
    RV::unpack(b, o);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += o[i];
    return RV::pack(v);
  };
  auto take = [&](int c, const typename RV::Raw& r) {
    if (hout.p) RV::store(hout.at(t) + c, r);
    float v[V], g[V];
    RV::unpack(r, v);
    if (Q) load_gain<V>(gain, c, g);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ss = fmaf(v[i], v[i], ss);
      if (Q) mx = max_nan(mx, fabsf(v[i] * g[i]));
    }
  };
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (c0 + j * step < H) {
      keep[j] = RV::load_rw(x.at(t) + c0 + j * step);
      if (res.p) add[j] = RV::load_rw(res.at(t) + c0 + j * step);
    }
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (c0 + j * step < H) {
      if (res.p) keep[j] = sum(keep[j], add[j]);
      take(c0 + j * step, keep[j]);
    }
  auto again = [&](int c) {
    const typename RV::Raw r = RV::load_rw(x.at(t) + c);
    return res.p ? sum(r, RV::load_rw(res.at(t) + c)) : r;
  };
  for (int c = c0 + NV * step; c < H; c += step) take(c, again(c));
  row_reduce<G, true>(ss, mx, part);
  const float r = 1.0f / sqrtf(ss / (float)H + eps);
  const float sc = max_nan(r * mx * (1.0f / kE4m3Max), kMinScale), inv = 1.0f / sc;
  const float ri = Q && sc > kMinScale ? r * inv : r, last = Q && !(sc > kMinScale) ? inv : 1.f;   // r * inv stays finite
  if (Q && tid == 0) scale[t] = sc;
  auto give = [&](int c, const typename RV::Raw& raw) {
    float v[V], g[V];
    RV::unpack(raw, v);
    load_gain<V>(gain, c, g);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = v[i] * g[i] * ri;
      if (Q && last != 1.f) v[i] *= last;
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
  for (int c = c0 + NV * step; c < H; c += step) give(c, hout.p ? RV::load_rw(hout.at(t) + c) : again(c));
}

// Rows blockIdx.x, + gridDim.x, ...  A thread keeps its columns: up to NV units of the row and of
// the gain's gradient stay in its registers; every block leaves the sum of grad_y * n over its
// rows in its row of `partial` [gridDim.x, H].  Bound by memory, so with NV <= 2 the next row is
// asked for before this one is reduced.  WIDE: columns behind the NV units are read again, and
// added up in `partial`.
template <typename T, int V, int NV, bool WIDE>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512, 1)
    rms_norm_backward_kernel(Rows<const T> gy, Rows<const T> h, const float* __restrict__ gain, float eps, int T_, int H,
                             Rows<const T> gh, Rows<T> gx, float* __restrict__ partial) {
  using RV = RowVec<T, V>;
  constexpr bool kAhead = NV <= 2 && !WIDE;
  __shared__ float2 part[32];
  ops_begin();
  float* mine = partial ? partial + (size_t)blockIdx.x * H : nullptr;
  const int step = blockDim.x * V, c0 = threadIdx.x * V;
  struct Row {
    typename RV::Raw g[NV], h[NV], e[NV];
  };
  auto load = [&](Row& r, long long t) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c0 + j * step < H && t < T_) {
        r.g[j] = RV::load(gy.at(t) + c0 + j * step);
        r.h[j] = RV::load(h.at(t) + c0 + j * step);
        if (gh.p) r.e[j] = RV::load_rw(gh.at(t) + c0 + j * step);
      }
  };
  float acc[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[j][i] = 0.f;
  Row now, next;
  load(now, blockIdx.x);
  for (long long t = blockIdx.x; t < T_; t += gridDim.x) {
    if (kAhead) load(next, t + gridDim.x);
    float ss = 0.f, su = 0.f;
    auto take = [&](int c, const typename RV::Raw& rg, const typename RV::Raw& rh) {
      float d[V], v[V], g[V];
      RV::unpack(rg, d);
      RV::unpack(rh, v);
      load_gain<V>(gain, c, g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ss = fmaf(v[i], v[i], ss);
        su = fmaf(d[i] * g[i], v[i], su);
      }
    };
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c0 + j * step < H) take(c0 + j * step, now.g[j], now.h[j]);
    if (WIDE)
      for (int c = c0 + NV * step; c < H; c += step) take(c, RV::load(gy.at(t) + c), RV::load(h.at(t) + c));
    row_reduce<0, false>(ss, su, part);
    const float r = 1.0f / sqrtf(ss / (float)H + eps);
    const float m = r * (su / (float)H);             // mean(u n)
    auto give = [&](int c, const typename RV::Raw& rg, const typename RV::Raw& rh, const typename RV::Raw& re, float (&dg)[V]) {
      float d[V], v[V], g[V], e[V], o[V];
      RV::unpack(rg, d);
      RV::unpack(rh, v);
      if (gh.p) RV::unpack(re, e);
      load_gain<V>(gain, c, g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float n = v[i] * r;
        o[i] = r * (d[i] * g[i] - n * m);
        if (gh.p) o[i] += e[i];
        dg[i] = fmaf(d[i], n, dg[i]);
      }
      RV::store(gx.at(t) + c, RV::pack(o));
    };
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c0 + j * step < H) give(c0 + j * step, now.g[j], now.h[j], now.e[j], acc[j]);
    if (WIDE)
      for (int c = c0 + NV * step; c < H; c += step) {
        float dg[V];
#pragma unroll
        for (int i = 0; i < V; ++i) dg[i] = mine && t != blockIdx.x ? mine[c + i] : 0.f;
        const typename RV::Raw rg = RV::load(gy.at(t) + c);
        give(c, rg, RV::load(h.at(t) + c), gh.p ? RV::load_rw(gh.at(t) + c) : rg, dg);
        if (mine) {
#pragma unroll
          for (int i = 0; i < V; ++i) mine[c + i] = dg[i];
        }
      }
    if (kAhead)
      now = next;
    else
      load(now, t + gridDim.x);
  }
  if (mine) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c0 + j * step < H) mine[c0 + j * step + i] = acc[j][i];
  }
}

// out[c] = sum over G rows of partial: 32 columns a block, 32 groups of rows, joined in order.
__global__ void __launch_bounds__(1024) sum_partials_kernel(const float* __restrict__ partial, int G, int H,
                                                            float* __restrict__ out) {
  __shared__ float sum[32][33];
  ops_begin();
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < H) {
#pragma unroll 4
    for (int g = grp; g < G; g += 32) a += partial[(size_t)g * H + c];
  }
  sum[grp][lane] = a;
  __syncthreads();
  a = warp_sum(sum[lane][grp]);                      // warp `grp`: column grp of the block
  if (lane == 0 && blockIdx.x * 32 + grp < H) out[blockIdx.x * 32 + grp] = a;
}

// Units a thread keeps, and threads: a warp takes a row of up to 64 units; a block has at most 256
// threads of up to 4 units where that holds the row, else as many as there may be.
template <typename T, int V, bool Q>
moe_status norm_launch(const Rows<const T>& x, const Rows<const T>& res, const float* gain, float eps, int T_, int H,
                       const Rows<T>& h, const Rows<T>& y, const Rows<uint8_t>& q, float* scale, void* s) {
  const int units = (H + V - 1) / V;
  if (units <= 64)
    return launch_op(add_rms_norm_kernel<T, V, 2, 32, Q>, dim3((unsigned)((T_ + 3LL) / 4)), 128, 0, 1, s, x, res, gain, eps,
                     T_, H, h, y, q, scale);
  const int most = V == 1 ? 1024 : 512;
  const int threads = std::min(most, ((units + 3) / 4 + 31) & ~31);
  return launch_op(add_rms_norm_kernel<T, V, 4, 0, Q>, dim3(T_), threads, 0, 1, s, x, res, gain, eps, T_, H, h, y, q,
                   scale);
}

template <typename T>
moe_status norm_dispatch(const void* x, int64_t ldx, const void* res, int64_t ldr, const float* gain, float eps, int T_,
                         int H, void* h, int64_t ldh, void* y, int64_t ldy, float* scale, void* s) {
  constexpr int N = Vec<T>::N;
  const Rows<const T> xr{static_cast<const T*>(x), ldx}, rr{static_cast<const T*>(res), ldr};
  const Rows<T> hr{static_cast<T*>(h), ldh};
  const Rows<T> yr{scale ? nullptr : static_cast<T*>(y), ldy};
  const Rows<uint8_t> qr{scale ? static_cast<uint8_t*>(y) : nullptr, ldy};
  const bool wide = H % N == 0 && rows16(x, ldx, sizeof(T)) && rows16(res, ldr, sizeof(T)) && rows16(h, ldh, sizeof(T)) &&
                    aligned16(gain);
  if (scale) {
    if (wide && reinterpret_cast<uintptr_t>(y) % N == 0 && ldy % N == 0)
      return norm_launch<T, N, true>(xr, rr, gain, eps, T_, H, hr, yr, qr, scale, s);
    return norm_launch<T, 1, true>(xr, rr, gain, eps, T_, H, hr, yr, qr, scale, s);
  }
  if (wide && rows16(y, ldy, sizeof(T)))
    return norm_launch<T, N, false>(xr, rr, gain, eps, T_, H, hr, yr, qr, scale, s);
  return norm_launch<T, 1, false>(xr, rr, gain, eps, T_, H, hr, yr, qr, scale, s);
}

// Blocks of the backward pass, the rows of `partial`: one an SM for rows of 8192 columns, more where
// they are short.
int norm_bwd_blocks(int T_, int H) { return std::min(T_, 152 * std::max(1, std::min(16, 9216 / H))); }

template <typename T, int V>
moe_status norm_backward_launch(int G, const Rows<const T>& gy, const Rows<const T>& h, const float* gain, float eps, int T_,
                                int H, const Rows<const T>& gh, const Rows<T>& gx, float* partial, void* s) {
  const int units = (H + V - 1) / V, most = V == 1 ? 1024 : 512;
  const int nv = units <= 128 ? 1 : units <= 2 * most ? 2 : 4;
  const int threads = std::min(most, ((units + nv - 1) / nv + 31) & ~31);
  auto go = [&](auto kernel) {
    return launch_op(kernel, dim3(G), threads, 0, 1, s, gy, h, gain, eps, T_, H, gh, gx, partial);
  };
  if (units > 4 * most) return go(rms_norm_backward_kernel<T, V, 2, true>);
  if (nv == 1) return go(rms_norm_backward_kernel<T, V, 1, false>);
  if (nv == 2) return go(rms_norm_backward_kernel<T, V, 2, false>);
  return go(rms_norm_backward_kernel<T, V, 4, false>);
}

template <typename T>
moe_status norm_backward_dispatch(const void* gy, int64_t ldgy, const void* h, int64_t ldh, const float* gain, float eps,
                                  int T_, int H, const void* gh, int64_t ldgh, void* gx, int64_t ldgx, float* ggain,
                                  float* ws, void* s) {
  constexpr int N = Vec<T>::N;
  const Rows<const T> a{static_cast<const T*>(gy), ldgy}, b{static_cast<const T*>(h), ldh},
      c{static_cast<const T*>(gh), ldgh};
  const Rows<T> o{static_cast<T*>(gx), ldgx};
  const int G = norm_bwd_blocks(T_, H);
  float* partial = ggain ? ws : nullptr;
  const bool wide = H % N == 0 && rows16(gy, ldgy, sizeof(T)) && rows16(h, ldh, sizeof(T)) &&
                    rows16(gh, ldgh, sizeof(T)) && rows16(gx, ldgx, sizeof(T)) && aligned16(gain);
  const moe_status st = wide ? norm_backward_launch<T, N>(G, a, b, gain, eps, T_, H, c, o, partial, s)
                             : norm_backward_launch<T, 1>(G, a, b, gain, eps, T_, H, c, o, partial, s);
  if (st != MOE_OK || !ggain) return st;
  return launch_op(sum_partials_kernel, dim3((H + 31) / 32), 1024, 0, 1, s, (const float*)ws, G, H, ggain);
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
  return T < 1 || H < 1 ? 0 : (int64_t)norm_bwd_blocks(T, H) * H * (int64_t)sizeof(float);
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
