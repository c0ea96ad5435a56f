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
#include <cmath>
#include "moe_ops.cuh"
#include "moe_ptx.cuh"

namespace moe {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;         // 2^-126

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum of a and NaN-keeping maximum of b over the G threads of a row (32, or the whole block), the
// same values in every thread.
template <int G>
__device__ __forceinline__ void row_sum_max(float& a, float& b, float2* part) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, off);
    b = max_nan(b, __shfl_xor_sync(0xffffffffu, b, off));
  }
  if (G == 32) return;
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < warps ? part[lane] : make_float2(0.f, 0.f);
  a = v.x;
  b = v.y;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, off);
    b = max_nan(b, __shfl_xor_sync(0xffffffffu, b, off));
  }
}

// Four sums over the block at once, the same in every thread: the lanes hand each other half of
// their values at a time, 6 shuffles instead of 20, and share the warps' sums alike.
__device__ __forceinline__ void block_sum4(float (&v)[4], float (*part)[4]) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const bool hi = lane & 16, odd = lane & 8;
  float a = hi ? v[2] : v[0], b = hi ? v[3] : v[1];
  a += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
  b += __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 16);
  float c = odd ? b : a;
  c += __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) c += __shfl_xor_sync(0xffffffffu, c, off);
  __syncthreads();                                   // `part` may still be read for the rows before
  if ((lane & 7) == 0) part[threadIdx.x >> 5][lane >> 3] = c;
  __syncthreads();
  c = 0.f;
  for (int w = lane >> 2; w < warps; w += 8) c += part[w][lane & 3];
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) c += __shfl_xor_sync(0xffffffffu, c, off);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, c, i);
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
__global__ void __launch_bounds__(G == 32 ? 128 : V == 1 ? 1024 : 512, G == 32 ? 8 : V == 1 ? 1 : 2)
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
  row_sum_max<G>(ss, mx, part);
  const float r = 1.0f / sqrtf(ss / (float)H + eps);
  // a sum or a product beyond fp32 (or NaN): r is 0 or the scale infinite, and zeros in 8 bits would hide it
  const bool lost = !(ss < INFINITY && r * mx < INFINITY);
  const float sc = lost ? NAN : fmaxf(r * mx * (1.0f / kE4m3Max), kMinScale), inv = 1.0f / sc;
  if (Q && tid == 0) scale[t] = sc;
  auto give = [&](int c, const typename RV::Raw& raw) {
    float v[V], g[V];
    RV::unpack(raw, v);
    load_gain<V>(gain, c, g);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // step by step, h / rms first, which is at most sqrt(H): h gain may pass fp32 where y does not, and so may r / scale
      // as one factor, 448 / max|h gain|.  1 / scale (at most 2^126) is taken once: a quotient per value took 42 us
      // for 4096 x 7168, 36 so.
      v[i] = v[i] * r * g[i];
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
  for (int c = c0 + NV * step; c < H; c += step) give(c, hout.p ? RV::load_rw(hout.at(t) + c) : again(c));
}

// Rows blockIdx.x, + gridDim.x, ..., two at a time.  A thread keeps its columns: up to NV units of
// the rows and of the gain's gradient stay in its registers; every block leaves the sum of
// grad_y * n over its rows in its row of `partial` [gridDim.x, H].  Bound by memory, and close
// behind by the instructions between a row's reads and its writes: hence two rows in flight and
// one reduction for both (one row at a time: 8192 x 2880 in 60 us, asking for the next one ahead
// 58).  WIDE: columns behind the NV units are read again, and added up in `partial`.
template <typename T, int V, int NV, bool WIDE, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 384 ? 3 : 1)
    rms_norm_backward_kernel(Rows<const T> gy, Rows<const T> h, const float* __restrict__ gain, float eps, int T_, int H,
                             Rows<const T> gh, Rows<T> gx, float* __restrict__ partial) {
  using RV = RowVec<T, V>;
  using Raw = typename RV::Raw;
  __shared__ float part[32][4];
  ops_begin();
  float* mine = partial ? partial + (size_t)blockIdx.x * H : nullptr;
  const int step = blockDim.x * V, c0 = threadIdx.x * V;
  float acc[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[j][i] = 0.f;
  for (long long t0 = blockIdx.x; t0 < T_; t0 += 2LL * gridDim.x) {
    Raw kg[2][NV], kh[2][NV], ke[2][NV];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const long long t = t0 + k * gridDim.x;
        const int c = c0 + j * step;
        if (c < H && t < T_) {
          kg[k][j] = RV::load(gy.at(t) + c);
          kh[k][j] = RV::load(h.at(t) + c);
          if (gh.p) ke[k][j] = RV::load_rw(gh.at(t) + c);
        }
      }
    float s[4] = {0.f, 0.f, 0.f, 0.f};               // per row: sum of h^2, sum of u h
    auto take = [&](int k, const float (&g)[V], const Raw& rg, const Raw& rh) {
      float d[V], v[V];
      RV::unpack(rg, d);
      RV::unpack(rh, v);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[2 * k] = fmaf(v[i], v[i], s[2 * k]);
        s[2 * k + 1] = fmaf(d[i] * g[i], v[i], s[2 * k + 1]);
      }
    };
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c0 + j * step < H) {
        float g[V];
        load_gain<V>(gain, c0 + j * step, g);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (t0 + k * gridDim.x < T_) take(k, g, kg[k][j], kh[k][j]);
      }
    if (WIDE)
      for (int c = c0 + NV * step; c < H; c += step) {
        float g[V];
        load_gain<V>(gain, c, g);
        for (int k = 0; k < 2; ++k) {
          const long long t = t0 + k * gridDim.x;
          if (t < T_) take(k, g, RV::load(gy.at(t) + c), RV::load(h.at(t) + c));
        }
      }
    block_sum4(s, part);
    float r[2], m[2];                                // 1 / rms (its square may pass fp32) and mean(u n)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      r[k] = 1.0f / sqrtf(s[2 * k] / (float)H + eps);
      m[k] = r[k] * s[2 * k + 1] / (float)H;
    }
    auto give = [&](int k, int c, const float (&g)[V], const Raw& rg, const Raw& rh, const Raw& re, float (&dg)[V]) {
      float d[V], v[V], e[V], o[V];
      RV::unpack(rg, d);
      RV::unpack(rh, v);
      if (gh.p) RV::unpack(re, e);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float n = v[i] * r[k];
        o[i] = r[k] * (d[i] * g[i] - n * m[k]);
        if (gh.p) o[i] += e[i];
        dg[i] = fmaf(d[i], n, dg[i]);
      }
      RV::store(gx.at(t0 + k * gridDim.x) + c, RV::pack(o));
    };
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c0 + j * step < H) {
        float g[V];
        load_gain<V>(gain, c0 + j * step, g);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (t0 + k * gridDim.x < T_) give(k, c0 + j * step, g, kg[k][j], kh[k][j], ke[k][j], acc[j]);
      }
    if (WIDE)
      for (int c = c0 + NV * step; c < H; c += step) {
        float g[V], dg[V];
        load_gain<V>(gain, c, g);
#pragma unroll
        for (int i = 0; i < V; ++i) dg[i] = mine && t0 != blockIdx.x ? mine[c + i] : 0.f;
        for (int k = 0; k < 2; ++k) {
          const long long t = t0 + k * gridDim.x;
          if (t >= T_) break;
          const Raw rg = RV::load(gy.at(t) + c);
          give(k, c, g, rg, RV::load(h.at(t) + c), gh.p ? RV::load_rw(gh.at(t) + c) : rg, dg);
        }
        if (mine) {
#pragma unroll
          for (int i = 0; i < V; ++i) mine[c + i] = dg[i];
        }
      }
  }
  if (mine) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c0 + j * step < H) mine[c0 + j * step + i] = acc[j][i];
  }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The same for rows of at most 1024 16-byte units: one unit a thread, which copies it for the next
// two rows into its own slots of shared memory while it works on these (no barrier: nobody else
// reads them), so every SM keeps reading, and holds no operand in registers across the reduction.
template <typename T>
__global__ void __launch_bounds__(1024, 1)
    rms_norm_backward_ring_kernel(Rows<const T> gy, Rows<const T> h, const float* __restrict__ gain, float eps, int T_, int H,
                                  Rows<const T> gh, Rows<T> gx, float* __restrict__ partial) {
  constexpr int V = Vec<T>::N;
  using RV = RowVec<T, V>;
  extern __shared__ uint4 slots[];                   // [2 stages][2 rows][grad_y, h, grad_h][thread]
  __shared__ float part[32][4];
  ops_begin();
  const int c = threadIdx.x * V;
  const bool live = c < H;
  auto slot = [&](int stage, int k, int o) { return slots + ((stage * 2 + k) * 3 + o) * blockDim.x + threadIdx.x; };
  auto fetch = [&](int stage, long long t0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long t = t0 + k * (long long)gridDim.x;
      if (live && t < T_) {
        copy16(ptx::smem_u32(slot(stage, k, 0)), gy.at(t) + c);
        copy16(ptx::smem_u32(slot(stage, k, 1)), h.at(t) + c);
        if (gh.p) copy16(ptx::smem_u32(slot(stage, k, 2)), gh.at(t) + c);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float acc[V], g[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  if (live) load_gain<V>(gain, c, g);
  int stage = 0;
  fetch(0, blockIdx.x);
  for (long long t0 = blockIdx.x; t0 < T_; t0 += 2LL * gridDim.x, stage ^= 1) {
    fetch(stage ^ 1, t0 + 2LL * gridDim.x);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    float s[4] = {0.f, 0.f, 0.f, 0.f};               // per row: sum of h^2, sum of u h
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (live && t0 + k * (long long)gridDim.x < T_) {
        float d[V], v[V];
        RV::unpack(*slot(stage, k, 0), d);
        RV::unpack(*slot(stage, k, 1), v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s[2 * k] = fmaf(v[i], v[i], s[2 * k]);
          s[2 * k + 1] = fmaf(d[i] * g[i], v[i], s[2 * k + 1]);
        }
      }
    block_sum4(s, part);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long t = t0 + k * (long long)gridDim.x;
      const float r = 1.0f / sqrtf(s[2 * k] / (float)H + eps);
      const float m = r * s[2 * k + 1] / (float)H;            // mean(u n); r * r may pass fp32
      if (live && t < T_) {
        float d[V], v[V], e[V], o[V];
        RV::unpack(*slot(stage, k, 0), d);
        RV::unpack(*slot(stage, k, 1), v);
        if (gh.p) RV::unpack(*slot(stage, k, 2), e);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float n = v[i] * r;
          o[i] = r * (d[i] * g[i] - n * m);
          if (gh.p) o[i] += e[i];
          acc[i] = fmaf(d[i], n, acc[i]);
        }
        RV::store(gx.at(t) + c, RV::pack(o));
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (partial && live) {
#pragma unroll
    for (int i = 0; i < V; ++i) partial[(size_t)blockIdx.x * H + c + i] = acc[i];
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
    for (int g0 = grp; g0 < G; g0 += 32 * 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = g0 + 32 * u < G ? __ldg(partial + (size_t)(g0 + 32 * u) * H + c) : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) a += v[u];
    }
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
// they are short.  152 is written out: the workspace's size is asked without a device, and the order of
// the gain's sums depends on sizes only.
int norm_bwd_blocks(int T_, int H) { return std::min(T_, 152 * std::max(1, std::min(8, 9216 / H))); }

template <typename T, int V>
moe_status norm_backward_launch(int G, const Rows<const T>& gy, const Rows<const T>& h, const float* gain, float eps, int T_,
                                int H, const Rows<const T>& gh, const Rows<T>& gx, float* partial, void* s) {
  const int units = (H + V - 1) / V;
  const int threads = units <= 1024 ? (units + 31) & ~31 : 512;
  auto go = [&](auto kernel) {
    return launch_op(kernel, dim3(G), threads, 0, 1, s, gy, h, gain, eps, T_, H, gh, gx, partial);
  };
  if constexpr (V > 1) {
    if (units <= 1024) {
      const size_t smem = (size_t)12 * 16 * threads;
      if (cudaFuncSetAttribute(rms_norm_backward_ring_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 12 * 16 * 1024) !=
          cudaSuccess)
        return MOE_ERR_CUDA;
      return launch_op(rms_norm_backward_ring_kernel<T>, dim3(G), threads, smem, 1, s, gy, h, gain, eps, T_, H, gh, gx, partial);
    }
    return go(rms_norm_backward_kernel<T, V, 2, true, 512>);        // four units spill
  } else {
    if (units <= 384) return go(rms_norm_backward_kernel<T, V, 1, false, 384>);    // three blocks an SM
    if (units <= 1024) return go(rms_norm_backward_kernel<T, V, 1, false, 1024>);
    if (units <= 2048) return go(rms_norm_backward_kernel<T, V, 4, false, 512>);
    return go(rms_norm_backward_kernel<T, V, 4, true, 512>);
  }
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
  if ((dtype != MOE_F32 && dtype != MOE_BF16) || T < 0 || H < 1 || H > kMaxWidth || !(eps >= 0.f)) return MOE_ERR_INVALID;
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
  if ((dtype != MOE_F32 && dtype != MOE_BF16) || T < 0 || H < 1 || H > kMaxWidth || !(eps >= 0.f)) return MOE_ERR_INVALID;
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
