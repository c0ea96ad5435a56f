// The synchronous dispatch of a routed batch: token rows sorted by expert, expert results merged
// back under the routing weights, and the gradients of both and of the router's weights.
//
//   pos[t, k]  row of pair (t, k) in the sorted order, -1 where its expert id is outside [0, E)
//   rows[pos[t, k]] = x[t]                               sort_rows
//   y[t] = sum_k w[t, k] rows[pos[t, k]] (+ residual[t])  merge_rows ("SOSP'26 StreamEP" section 3)
//   grad_rows[pos[t, k]] = w[t, k] grad_y[t],  grad_w[t, k] = <rows[pos[t, k]], grad_y[t]>
//   grad_x[t] = sum_k grad_rows[pos[t, k]]               merge_rows without weights
//   grad_logit[t, idx_k] = w_k (grad_w_k - sum_j w_j grad_w_j)
//
// The order is stable (by expert, then by pair t K + k), so it, and every sum taken along it,
// is the same on every run: no float atomics anywhere.
#include <algorithm>
#include "moe_ops.cuh"

namespace moe {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;

// ------------------------------------------------------------------ sort_experts

// One block, a stable counting sort: every warp owns a contiguous range of pairs and a histogram
// of its own; an exclusive scan over (expert, warp) turns the histograms into first positions;
// the warps walk their ranges again and hand out positions in pair order.  Bucket E holds the
// pairs that belong to no expert here, behind all others.
__global__ void __launch_bounds__(kSortThreads) sort_experts_kernel(const int32_t* __restrict__ expert, int P, int E,
                                                                    int32_t* __restrict__ offsets,
                                                                    int32_t* __restrict__ pos,
                                                                    int32_t* __restrict__ pair) {
  extern __shared__ int hist[];                      // [warps][E + 1]
  __shared__ int wsum[kSortWarps];
  const int NB = E + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * NB; i += kSortThreads) hist[i] = 0;
  ops_begin();
  __syncthreads();
  const int per = ((P + kSortWarps - 1) / kSortWarps + 31) & ~31;
  const long long p0 = (long long)warp * per;
  const long long p1 = min((long long)P, p0 + per);
  int* h = hist + warp * NB;
  for (long long i = p0 + lane; i < p1; i += 32) {
    const int e = expert[i];
    atomicAdd(&h[e >= 0 && e < E ? e : E], 1);
  }
  __syncthreads();
  // exclusive scan in (bucket, warp) order: two buckets a thread cover 1025 of them
  int tot[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int b = 2 * threadIdx.x + u;
    int s = 0;
    if (b < NB)
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = hist[w * NB + b];
        hist[w * NB + b] = s;
        s += c;
      }
    tot[u] = s;
  }
  int s = tot[0] + tot[1], incl = s;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int start = incl - s;
  for (int w = 0; w < warp; ++w) start += wsum[w];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int b = 2 * threadIdx.x + u;
    if (b < NB) {
      for (int w = 0; w < kSortWarps; ++w) hist[w * NB + b] += start;
      offsets[b] = start;                           // bucket E starts where the last expert ends
    }
    start += tot[u];
  }
  __syncthreads();
  for (long long i0 = p0; i0 < p1; i0 += 32) {
    const long long i = i0 + lane;
    const int e = i < p1 ? expert[i] : -2;
    const int b = i < p1 ? (e >= 0 && e < E ? e : E) : NB;
    const unsigned same = __match_any_sync(0xffffffffu, b);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int base = 0;
    if (i < p1) base = h[b];
    __syncwarp();
    if (i < p1 && rank == 0) h[b] = base + __popc(same);
    __syncwarp();
    if (i < p1) {
      pos[i] = b < E ? base + rank : -1;
      pair[base + rank] = (int)i;
    }
  }
}

// ------------------------------------------------------------------ sort_rows

constexpr int kRowThreads = 256;

// Block (t, part): its part of token t's row, read once and written to the rows of its pairs.
template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) sort_rows_kernel(Rows<const T> x, const int32_t* __restrict__ pos, int K,
                                                                int H, long long R, Rows<T> rows) {
  using RV = RowVec<T, V>;
  ops_begin();
  const long long t = blockIdx.x;
  const int32_t* pt = pos + t * K;
  const T* src = x.at(t);
  for (int c = (blockIdx.y * kRowThreads + threadIdx.x) * V; c < H; c += gridDim.y * kRowThreads * V) {
    const typename RV::Raw v = RV::load(src + c);
    for (int k = 0; k < K; ++k) {
      const int p = __ldg(pt + k);
      if (p >= 0 && p < R) RV::store(rows.at(p) + c, v);
    }
  }
}

// ------------------------------------------------------------------ merge_rows

// Block (t, part): products and sums rounded in fp32 in ascending k, as in the collect kernel,
// then the residual; rounded to T once.  w == nullptr: plain sum.
template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) merge_rows_kernel(Rows<const T> rows, long long R,
                                                                 const int32_t* __restrict__ pos,
                                                                 const float* __restrict__ w, int K, int H,
                                                                 Rows<const T> residual, Rows<T> y) {
  using RV = RowVec<T, V>;
  ops_begin();
  const long long t = blockIdx.x;
  const int32_t* pt = pos + t * K;
  for (int c = (blockIdx.y * kRowThreads + threadIdx.x) * V; c < H; c += gridDim.y * kRowThreads * V) {
    float a[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = 0.f;
    for (int k = 0; k < K; ++k) {
      const int p = __ldg(pt + k);
      if (p < 0 || p >= R) continue;
      float v[V];
      RV::unpack(RV::load(rows.at(p) + c), v);
      const float wk = w ? __ldg(w + t * K + k) : 1.f;
#pragma unroll
      for (int i = 0; i < V; ++i) a[i] = __fadd_rn(a[i], __fmul_rn(wk, v[i]));
    }
    if (residual.p) {
      float v[V];
      RV::unpack(RV::load_rw(residual.at(t) + c), v);
#pragma unroll
      for (int i = 0; i < V; ++i) a[i] = __fadd_rn(a[i], v[i]);
    }
    RV::store(y.at(t) + c, RV::pack(a));
  }
}

// Block t: grad_rows of its pairs and grad_w, kMergeK pairs at a time.
constexpr int kMergeK = 8;
template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads)
    merge_rows_backward_kernel(Rows<const T> grad, Rows<const T> rows, long long R, const int32_t* __restrict__ pos,
                               const float* __restrict__ w, int K, int H, Rows<T> grad_rows,
                               float* __restrict__ grad_w) {
  using RV = RowVec<T, V>;
  __shared__ float part[kRowThreads / 32][kMergeK];
  ops_begin();
  const long long t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int k0 = 0; k0 < K; k0 += kMergeK) {
    int p[kMergeK];
    float wk[kMergeK], dot[kMergeK];
#pragma unroll
    for (int u = 0; u < kMergeK; ++u) {
      p[u] = k0 + u < K ? __ldg(pos + t * K + k0 + u) : -1;
      if (p[u] >= R) p[u] = -1;
      wk[u] = k0 + u < K ? __ldg(w + t * K + k0 + u) : 0.f;
      dot[u] = 0.f;
    }
    for (int c = threadIdx.x * V; c < H; c += kRowThreads * V) {
      float g[V];
      RV::unpack(RV::load(grad.at(t) + c), g);
#pragma unroll
      for (int u = 0; u < kMergeK; ++u) {
        if (p[u] >= 0) {
          float v[V], o[V];
          RV::unpack(RV::load(rows.at(p[u]) + c), v);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            dot[u] = fmaf(v[i], g[i], dot[u]);
            o[i] = wk[u] * g[i];
          }
          RV::store(grad_rows.at(p[u]) + c, RV::pack(o));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kMergeK; ++u) {
      const float d = warp_sum(dot[u]);
      if (lane == 0) part[warp][u] = d;
    }
    __syncthreads();
    if (threadIdx.x < kMergeK && k0 + threadIdx.x < K) {
      float d = 0.f;
      for (int i = 0; i < kRowThreads / 32; ++i) d += part[i][threadIdx.x];
      grad_w[t * K + k0 + threadIdx.x] = d;
    }
    __syncthreads();
  }
}

// One warp per token: lane k holds pair k (K <= 32); every expert's column adds the pairs that
// chose it in ascending k.
__global__ void route_backward_kernel(const int32_t* __restrict__ idx, const float* __restrict__ w,
                                      const float* __restrict__ grad_w, int T, int E, int K,
                                      float* __restrict__ grad_logits) {
  ops_begin();
  const int lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= T) return;
  const int id = lane < K ? idx[t * K + lane] : -1;
  const float wk = lane < K ? w[t * K + lane] : 0.f, g = lane < K ? grad_w[t * K + lane] : 0.f;
  const float mean = warp_sum(wk * g);
  const float d = wk * (g - mean);
  float* out = grad_logits + t * E;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    float v = 0.f;
    for (int k = 0; k < K; ++k) {
      const int ik = __shfl_sync(0xffffffffu, id, k);
      const float dk = __shfl_sync(0xffffffffu, d, k);
      if (ik == e) v += dk;
    }
    if (e < E) out[e] = v;
  }
}

bool valid_rows(int32_t dtype, int32_t T, int32_t K, int32_t H, int64_t R) {
  return (dtype == MOE_F32 || dtype == MOE_BF16) && T >= 0 && K >= 1 && K <= 32 && H >= 1 && R >= 0 &&
         (int64_t)T * K <= INT32_MAX && R <= INT32_MAX;
}

// Blocks along a row: one covers kRowThreads vectors; few tokens spread their rows over more.
int row_parts(int H, int v) { return std::max(1, std::min(65535, (H + kRowThreads * v - 1) / (kRowThreads * v))); }

template <typename T>
moe_status sort_rows_launch(const void* x, int64_t ldx, const int32_t* pos, int T_, int K, int H, int64_t R, void* rows,
                            int64_t ldr, void* s) {
  constexpr int N = Vec<T>::N;
  const Rows<const T> in{static_cast<const T*>(x), ldx};
  const Rows<T> out{static_cast<T*>(rows), ldr};
  const long long r = R;
  if (H % N == 0 && rows16(x, ldx, sizeof(T)) && rows16(rows, ldr, sizeof(T)))
    return launch_op(sort_rows_kernel<T, N>, dim3(T_, row_parts(H, N)), kRowThreads, 0, 1, s, in, pos, K, H, r, out);
  return launch_op(sort_rows_kernel<T, 1>, dim3(T_, row_parts(H, 1)), kRowThreads, 0, 1, s, in, pos, K, H, r, out);
}

template <typename T>
moe_status merge_rows_launch(const void* rows, int64_t ldr, int64_t R, const int32_t* pos, const float* w, int T_, int K,
                             int H, const void* res, int64_t ldres, void* y, int64_t ldy, void* s) {
  constexpr int N = Vec<T>::N;
  const Rows<const T> in{static_cast<const T*>(rows), ldr}, add{static_cast<const T*>(res), ldres};
  const Rows<T> out{static_cast<T*>(y), ldy};
  const long long r = R;
  if (H % N == 0 && rows16(rows, ldr, sizeof(T)) && rows16(res, ldres, sizeof(T)) && rows16(y, ldy, sizeof(T)))
    return launch_op(merge_rows_kernel<T, N>, dim3(T_, row_parts(H, N)), kRowThreads, 0, 1, s, in, r, pos, w, K, H, add,
                     out);
  return launch_op(merge_rows_kernel<T, 1>, dim3(T_, row_parts(H, 1)), kRowThreads, 0, 1, s, in, r, pos, w, K, H, add,
                   out);
}

template <typename T>
moe_status merge_backward_launch(const void* grad, int64_t ldg, const void* rows, int64_t ldr, int64_t R,
                                 const int32_t* pos, const float* w, int T_, int K, int H, void* grows, int64_t ldgr,
                                 float* gw, void* s) {
  constexpr int N = Vec<T>::N;
  const Rows<const T> g{static_cast<const T*>(grad), ldg}, in{static_cast<const T*>(rows), ldr};
  const Rows<T> out{static_cast<T*>(grows), ldgr};
  const long long r = R;
  if (H % N == 0 && rows16(grad, ldg, sizeof(T)) && rows16(rows, ldr, sizeof(T)) && rows16(grows, ldgr, sizeof(T)))
    return launch_op(merge_rows_backward_kernel<T, N>, dim3(T_), kRowThreads, 0, 1, s, g, in, r, pos, w, K, H, out, gw);
  return launch_op(merge_rows_backward_kernel<T, 1>, dim3(T_), kRowThreads, 0, 1, s, g, in, r, pos, w, K, H, out, gw);
}

}  // namespace
}  // namespace moe

extern "C" {
using namespace moe;

moe_status moe_async_sort_experts(const int32_t* d_expert, int32_t T, int32_t K, int32_t E, int32_t* d_offsets,
                                  int32_t* d_pos, int32_t* d_pair, void* stream) {
  if (T < 0 || K < 1 || K > 32 || E < 1 || E > kMaxExperts || (int64_t)T * K > INT32_MAX - 1024) return MOE_ERR_INVALID;
  if (!d_offsets || (T > 0 && (!d_expert || !d_pos || !d_pair))) return MOE_ERR_INVALID;
  const size_t smem = (size_t)kSortWarps * (E + 1) * sizeof(int);
  if (smem > 48 * 1024 && cudaFuncSetAttribute(sort_experts_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem) != cudaSuccess)
    return MOE_ERR_CUDA;
  return launch_op(sort_experts_kernel, dim3(1), kSortThreads, smem, 1, stream, d_expert, T * K, E, d_offsets, d_pos,
                   d_pair);
}

moe_status moe_async_sort_rows(int32_t dtype, const void* d_x, int64_t x_stride, const int32_t* d_pos, int32_t T,
                               int32_t K, int32_t H, void* d_rows, int64_t rows_stride, int64_t n_rows, void* stream) {
  if (!valid_rows(dtype, T, K, H, n_rows)) return MOE_ERR_INVALID;
  if (T == 0 || n_rows == 0) return MOE_OK;
  if (!d_x || !d_pos || !d_rows || x_stride < H || rows_stride < H) return MOE_ERR_INVALID;
  return dtype == MOE_BF16
             ? sort_rows_launch<__nv_bfloat16>(d_x, x_stride, d_pos, T, K, H, n_rows, d_rows, rows_stride, stream)
             : sort_rows_launch<float>(d_x, x_stride, d_pos, T, K, H, n_rows, d_rows, rows_stride, stream);
}

moe_status moe_async_merge_rows(int32_t dtype, const void* d_rows, int64_t rows_stride, int64_t n_rows,
                                const int32_t* d_pos, const float* d_w, int32_t T, int32_t K, int32_t H,
                                const void* d_residual, int64_t residual_stride, void* d_y, int64_t y_stride,
                                void* stream) {
  if (!valid_rows(dtype, T, K, H, n_rows)) return MOE_ERR_INVALID;
  if (T == 0) return MOE_OK;
  if ((n_rows > 0 && (!d_rows || rows_stride < H)) || !d_pos || !d_y || y_stride < H ||
      (d_residual && residual_stride < H))
    return MOE_ERR_INVALID;
  return dtype == MOE_BF16 ? merge_rows_launch<__nv_bfloat16>(d_rows, rows_stride, n_rows, d_pos, d_w, T, K, H,
                                                              d_residual, residual_stride, d_y, y_stride, stream)
                           : merge_rows_launch<float>(d_rows, rows_stride, n_rows, d_pos, d_w, T, K, H, d_residual,
                                                      residual_stride, d_y, y_stride, stream);
}

moe_status moe_async_merge_rows_backward(int32_t dtype, const void* d_grad, int64_t grad_stride, const void* d_rows,
                                         int64_t rows_stride, int64_t n_rows, const int32_t* d_pos, const float* d_w,
                                         int32_t T, int32_t K, int32_t H, void* d_grad_rows, int64_t grad_rows_stride,
                                         float* d_grad_w, void* stream) {
  if (!valid_rows(dtype, T, K, H, n_rows)) return MOE_ERR_INVALID;
  if (T == 0) return MOE_OK;
  if (!d_grad || !d_pos || !d_w || !d_grad_w || grad_stride < H ||
      (n_rows > 0 && (!d_rows || !d_grad_rows || rows_stride < H || grad_rows_stride < H)))
    return MOE_ERR_INVALID;
  return dtype == MOE_BF16
             ? merge_backward_launch<__nv_bfloat16>(d_grad, grad_stride, d_rows, rows_stride, n_rows, d_pos, d_w, T, K,
                                                    H, d_grad_rows, grad_rows_stride, d_grad_w, stream)
             : merge_backward_launch<float>(d_grad, grad_stride, d_rows, rows_stride, n_rows, d_pos, d_w, T, K, H,
                                            d_grad_rows, grad_rows_stride, d_grad_w, stream);
}

moe_status moe_async_route_backward(const int32_t* d_idx, const float* d_w, const float* d_grad_w, int32_t T, int32_t E,
                                    int32_t K, float* d_grad_logits, void* stream) {
  if (T < 0 || E < 1 || E > kMaxExperts || K < 1 || K > E || K > 32) return MOE_ERR_INVALID;
  if (T == 0) return MOE_OK;
  if (!d_idx || !d_w || !d_grad_w || !d_grad_logits) return MOE_ERR_INVALID;
  return launch_op(route_backward_kernel, dim3((T + 7) / 8), 256, 0, 1, stream, d_idx, d_w, d_grad_w, T, E, K,
                   d_grad_logits);
}

}  // extern "C"
