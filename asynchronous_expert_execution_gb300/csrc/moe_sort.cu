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
#include "moe_ptx.cuh"

namespace moe {
namespace {

// ------------------------------------------------------------------ sort_experts

// A stable counting sort in one launch by one cluster of C CTAs.  Every warp owns a contiguous range
// of pairs and a histogram of its own; the scan over (expert, CTA, warp) turns the histograms into
// first positions, the CTAs' totals passing through distributed shared memory; the warps walk
// their ranges again and hand out positions in pair order.  Bucket E holds the pairs that belong
// to no expert here, behind all others.  Bound by latency (2 M pairs are 25 MB): eight loads are in
// flight per lane, and ranges of up to kKeep x 32 pairs stay in registers between the two walks.  Lanes of one
// expert find each other by ballots over the id's bits (524288 pairs: 86 us by matching whole ids, 61 so).
constexpr int kKeep = 8;
constexpr int kSortCluster = 8;
constexpr int kSortSmem = (32 + 3) * (kMaxExperts + 1) * (int)sizeof(int);       // of a block, at most

__global__ void __launch_bounds__(1024) sort_experts_kernel(const int32_t* __restrict__ expert, int P, int E, int per,
                                                            int32_t* __restrict__ offsets, int32_t* __restrict__ pos,
                                                            int32_t* __restrict__ pair) {
  extern __shared__ int sh[];
  __shared__ int wsum[32];
  const int NB = E + 1, warps = blockDim.x >> 5;
  int* hist = sh;                                    // [warps][E + 1]
  int* total = sh + warps * NB;                      // [E + 1] each: this CTA's pairs, all CTAs', first positions
  int* all = total + NB;
  int* first = all + NB;
  const int C = gridDim.x, rank = blockIdx.x;        // the grid is one cluster
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < warps * NB; i += blockDim.x) hist[i] = 0;
  ops_begin();
  __syncthreads();
  const long long p0 = min((long long)P, (long long)(rank * warps + warp) * per), p1 = min((long long)P, p0 + per);
  int* h = hist + warp * NB;
  auto bucket = [&](long long i) {
    const int e = i < p1 ? __ldg(expert + i) : -1;
    return e >= 0 && e < E ? e : E;
  };
  int keep[kKeep];                                   // the first kKeep x 32 of the range
  for (long long i0 = p0; i0 < p1; i0 += 32 * kKeep) {
    int b[kKeep];
#pragma unroll
    for (int u = 0; u < kKeep; ++u) b[u] = bucket(i0 + 32 * u + lane);
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
      if (i0 + 32 * u + lane < p1) atomicAdd(&h[b[u]], 1);
      if (i0 == p0) keep[u] = b[u];
    }
  }
  __syncthreads();
  // exclusive scan over the warps per bucket, and this CTA's totals
  for (int b = tid; b < NB; b += blockDim.x) {
    int s = 0;
    for (int w = 0; w < warps; ++w) {
      const int c = hist[w * NB + b];
      hist[w * NB + b] = s;
      s += c;
    }
    total[b] = s;
  }
  if (C > 1) ptx::cluster_sync(); else __syncthreads();
  for (int b = tid; b < NB; b += blockDim.x) {       // over all CTAs, and over those before this one
    int n[kSortCluster], sum = 0, before = 0;
#pragma unroll
    for (int r = 0; r < kSortCluster; ++r)
      n[r] = r < C ? (C > 1 ? ptx::ld_cluster_s32(ptx::mapa(ptx::smem_u32(total + b), r)) : total[b]) : 0;
#pragma unroll
    for (int r = 0; r < kSortCluster; ++r) {
      sum += n[r];
      if (r < rank) before += n[r];
    }
    all[b] = sum;
    first[b] = before;
  }
  if (C > 1) ptx::cluster_arrive();
  __syncthreads();
  // a bucket's first position: everything in the buckets before it, then its pairs of the CTAs before
  const int each = (NB + blockDim.x - 1) / blockDim.x;
  int mine = 0;
  for (int b = tid * each; b < min(NB, (tid + 1) * each); ++b) mine += all[b];
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int start = incl - mine;
  for (int w = 0; w < warp; ++w) start += wsum[w];
  for (int b = tid * each; b < min(NB, (tid + 1) * each); ++b) {
    if (rank == 0) offsets[b] = start;               // bucket E starts where the last expert ends
    first[b] += start;
    start += all[b];
  }
  __syncthreads();
  for (int b = tid; b < NB; b += blockDim.x)
    for (int w = 0; w < warps; ++w) hist[w * NB + b] += first[b];
  __syncthreads();
  const int bits = 32 - __clz(NB);
  for (long long i0 = p0; i0 < p1; i0 += 32 * kKeep) {
    int b[kKeep];
#pragma unroll
    for (int u = 0; u < kKeep; ++u) b[u] = i0 == p0 ? keep[u] : bucket(i0 + 32 * u + lane);
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
      const long long i = i0 + 32 * u + lane;
      if (i0 + 32 * u >= p1) break;
      const int key = i < p1 ? b[u] : NB;            // lanes behind the range form a group of their own
      unsigned same = 0xffffffffu;                   // lanes with this key, by the bits of the keys
      for (int bit = 0; bit < bits; ++bit) {
        const bool one = key >> bit & 1;
        const unsigned ones = __ballot_sync(0xffffffffu, one);
        same &= one ? ones : ~ones;
      }
      const int at = __popc(same & ((1u << lane) - 1u));
      const int base = i < p1 ? h[key] : 0;
      __syncwarp();
      if (i < p1 && at == 0) h[key] = base + __popc(same);
      __syncwarp();
      if (i < p1) {
        pos[i] = key < E ? base + at : -1;
        pair[base + at] = (int)i;
      }
    }
  }
  if (C > 1) ptx::cluster_wait();                    // no CTA ends while another reads its totals
}

// ------------------------------------------------------------------ sort_rows

constexpr int kRowThreads = 256;       // most threads of a block

// How rows lie on blocks: blockDim.x threads a row, blockDim.y rows a block (MANY: several, where rows
// are short), gridDim.y blocks a row where it is longer than 256 units.  With one row a block the row,
// its positions and its weights are the same for all threads, which the compiler uses: 2048 x 8 x
// 7168 merged in 48.8 us, 55.7 without.
template <bool MANY>
__device__ __forceinline__ long long row_of() {
  return MANY ? (long long)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
}

// A thread reads one unit of token t's row and writes it to the rows of its pairs.  Bound by the
// writes.
template <typename T, int V, bool MANY>
__global__ void __launch_bounds__(kRowThreads) sort_rows_kernel(Rows<const T> x, const int32_t* __restrict__ pos, int T_,
                                                                int K, int H, long long R, Rows<T> rows) {
  using RV = RowVec<T, V>;
  ops_begin();
  const long long t = row_of<MANY>();
  if (MANY && t >= T_) return;
  const int32_t* pt = pos + t * K;
  for (long long c = ((long long)blockIdx.y * blockDim.x + threadIdx.x) * V; c < H; c += (long long)gridDim.y * blockDim.x * V) {
    const typename RV::Raw v = RV::load(x.at(t) + c);
    for (int k = 0; k < K; ++k) {
      const int p = __ldg(pt + k);
      if (p >= 0 && p < R) RV::store(rows.at(p) + c, v);
    }
  }
}

// ------------------------------------------------------------------ merge_rows

// Products and sums rounded in fp32 in ascending k, as in the collect kernel,
// then the residual; rounded to T once.  w == nullptr: plain sum.  A thread owns one unit of the
// row and asks for KU result rows' units (and the residual's) before it uses the first.
template <typename T, int V, int KU, bool MANY>
__global__ void __launch_bounds__(kRowThreads) merge_rows_kernel(Rows<const T> rows, long long R,
                                                                 const int32_t* __restrict__ pos,
                                                                 const float* __restrict__ w, int T_, int K, int H,
                                                                 Rows<const T> residual, Rows<T> y) {
  using RV = RowVec<T, V>;
  ops_begin();
  const long long t = row_of<MANY>();
  if (MANY && t >= T_) return;
  for (long long c = ((long long)blockIdx.y * blockDim.x + threadIdx.x) * V; c < H; c += (long long)gridDim.y * blockDim.x * V) {
    float a[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = 0.f;
    typename RV::Raw last;
    if (residual.p) last = RV::load_rw(residual.at(t) + c);
    for (int k0 = 0; k0 < K; k0 += KU) {
      typename RV::Raw raw[KU];
      int p[KU];
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        p[u] = k0 + u < K ? __ldg(pos + t * K + k0 + u) : -1;
        if (p[u] >= R) p[u] = -1;
      }
#pragma unroll
      for (int u = 0; u < KU; ++u)
        if (p[u] >= 0) raw[u] = RV::load(rows.at(p[u]) + c);
#pragma unroll
      for (int u = 0; u < KU; ++u)
        if (p[u] >= 0) {
          float v[V];
          RV::unpack(raw[u], v);
          const float wk = w ? __ldg(w + t * K + k0 + u) : 1.f;
#pragma unroll
          for (int i = 0; i < V; ++i) a[i] = __fadd_rn(a[i], __fmul_rn(wk, v[i]));
        }
    }
    if (residual.p) {
      float v[V];
      RV::unpack(last, v);
#pragma unroll
      for (int i = 0; i < V; ++i) a[i] = __fadd_rn(a[i], v[i]);
    }
    RV::store(y.at(t) + c, RV::pack(a));
  }
}

// grad_rows of a token's pairs and grad_w, KU pairs at a time, all their reads in flight.
template <typename T, int V, int KU, bool MANY>
__global__ void __launch_bounds__(kRowThreads)
    merge_rows_backward_kernel(Rows<const T> grad, Rows<const T> rows, long long R, const int32_t* __restrict__ pos,
                               const float* __restrict__ w, int T_, int K, int H, Rows<T> grad_rows,
                               float* __restrict__ grad_w) {
  using RV = RowVec<T, V>;
  __shared__ float part[kRowThreads / 32][KU];
  ops_begin();
  const long long t = row_of<MANY>();
  const int warps = blockDim.x >> 5, row = MANY ? threadIdx.y : 0, warp = row * warps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  for (int k0 = 0; k0 < K; k0 += KU) {
    int p[KU];
    float wk[KU], dot[KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      p[u] = (!MANY || t < T_) && k0 + u < K ? __ldg(pos + t * K + k0 + u) : -1;
      if (p[u] >= R) p[u] = -1;
      wk[u] = (!MANY || t < T_) && k0 + u < K ? __ldg(w + t * K + k0 + u) : 0.f;
      dot[u] = 0.f;
    }
    for (int c = threadIdx.x * V; c < H && (!MANY || t < T_); c += blockDim.x * V) {
      const typename RV::Raw rg = RV::load(grad.at(t) + c);
      typename RV::Raw raw[KU];
#pragma unroll
      for (int u = 0; u < KU; ++u)
        if (p[u] >= 0) raw[u] = RV::load(rows.at(p[u]) + c);
      float g[V];
      RV::unpack(rg, g);
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        if (p[u] >= 0) {
          float v[V], o[V];
          RV::unpack(raw[u], v);
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
    for (int u = 0; u < KU; ++u) {
      const float d = warp_sum(dot[u]);
      if (lane == 0) part[warp][u] = d;
    }
    __syncthreads();
    if ((!MANY || t < T_) && threadIdx.x < KU && k0 + threadIdx.x < K) {
      float d = 0.f;
      for (int i = 0; i < warps; ++i) d += part[row * warps + i][threadIdx.x];
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
  return (dtype == MOE_F32 || dtype == MOE_BF16) && T >= 0 && K >= 1 && K <= 32 && H >= 1 && H <= kMaxWidth && R >= 0 &&
         (int64_t)T * K <= INT32_MAX && R <= INT32_MAX;
}

// A row's units over blocks of at most kRowThreads threads (whole warps a row).
struct RowGrid {
  dim3 grid, block;
  RowGrid(int T_, int H, int v, bool whole = false) {         // whole: one block takes all of a row
    const int units = (H + v - 1) / v;
    const int parts = std::min(65535, (units + kRowThreads - 1) / kRowThreads);
    block.x = std::min(kRowThreads, ((units + parts - 1) / parts + 31) & ~31);
    block.y = kRowThreads / block.x;
    grid.x = (unsigned)(((long long)T_ + block.y - 1) / block.y);
    grid.y = whole ? 1 : parts;
  }
  bool many() const { return block.y > 1; }
};

template <typename T, int V>
moe_status sort_rows_launch(const Rows<const T>& x, const int32_t* pos, int T_, int K, int H, long long R, const Rows<T>& rows,
                            void* s) {
  const RowGrid g(T_, H, V);
  auto go = [&](auto kernel) { return launch_op(kernel, g.grid, g.block, 0, 1, s, x, pos, T_, K, H, R, rows); };
  return g.many() ? go(sort_rows_kernel<T, V, true>) : go(sort_rows_kernel<T, V, false>);
}

template <typename T, int V>
moe_status merge_rows_launch(const Rows<const T>& rows, long long R, const int32_t* pos, const float* w, int T_, int K, int H,
                             const Rows<const T>& res, const Rows<T>& y, void* s) {
  const RowGrid g(T_, H, V);
  auto go = [&](auto kernel) { return launch_op(kernel, g.grid, g.block, 0, 1, s, rows, R, pos, w, T_, K, H, res, y); };
  if (g.many()) return K <= 4 ? go(merge_rows_kernel<T, V, 4, true>) : go(merge_rows_kernel<T, V, 8, true>);
  return K <= 4 ? go(merge_rows_kernel<T, V, 4, false>) : go(merge_rows_kernel<T, V, 8, false>);
}

template <typename T, int V>
moe_status merge_backward_launch(const Rows<const T>& grad, const Rows<const T>& rows, long long R, const int32_t* pos,
                                 const float* w, int T_, int K, int H, const Rows<T>& grad_rows, float* grad_w, void* s) {
  const RowGrid g(T_, H, V, true);
  auto go = [&](auto kernel) {
    return launch_op(kernel, g.grid, g.block, 0, 1, s, grad, rows, R, pos, w, T_, K, H, grad_rows, grad_w);
  };
  if (g.many()) return K <= 4 ? go(merge_rows_backward_kernel<T, V, 4, true>) : go(merge_rows_backward_kernel<T, V, 8, true>);
  return K <= 4 ? go(merge_rows_backward_kernel<T, V, 4, false>) : go(merge_rows_backward_kernel<T, V, 8, false>);
}

template <typename T>
moe_status sort_rows_dispatch(const void* x, int64_t ldx, const int32_t* pos, int T_, int K, int H, int64_t R, void* rows,
                              int64_t ldr, void* s) {
  constexpr int N = Vec<T>::N;
  const Rows<const T> in{static_cast<const T*>(x), ldx};
  const Rows<T> out{static_cast<T*>(rows), ldr};
  return H % N == 0 && rows16(x, ldx, sizeof(T)) && rows16(rows, ldr, sizeof(T))
             ? sort_rows_launch<T, N>(in, pos, T_, K, H, R, out, s)
             : sort_rows_launch<T, 1>(in, pos, T_, K, H, R, out, s);
}

template <typename T>
moe_status merge_rows_dispatch(const void* rows, int64_t ldr, int64_t R, const int32_t* pos, const float* w, int T_, int K,
                               int H, const void* res, int64_t ldres, void* y, int64_t ldy, void* s) {
  constexpr int N = Vec<T>::N;
  const Rows<const T> in{static_cast<const T*>(rows), ldr}, add{static_cast<const T*>(res), ldres};
  const Rows<T> out{static_cast<T*>(y), ldy};
  return H % N == 0 && rows16(rows, ldr, sizeof(T)) && rows16(res, ldres, sizeof(T)) && rows16(y, ldy, sizeof(T))
             ? merge_rows_launch<T, N>(in, R, pos, w, T_, K, H, add, out, s)
             : merge_rows_launch<T, 1>(in, R, pos, w, T_, K, H, add, out, s);
}

template <typename T>
moe_status merge_backward_dispatch(const void* grad, int64_t ldg, const void* rows, int64_t ldr, int64_t R,
                                   const int32_t* pos, const float* w, int T_, int K, int H, void* grows, int64_t ldgr,
                                   float* gw, void* s) {
  constexpr int N = Vec<T>::N;
  const Rows<const T> g{static_cast<const T*>(grad), ldg}, in{static_cast<const T*>(rows), ldr};
  const Rows<T> out{static_cast<T*>(grows), ldgr};
  return H % N == 0 && rows16(grad, ldg, sizeof(T)) && rows16(rows, ldr, sizeof(T)) && rows16(grows, ldgr, sizeof(T))
             ? merge_backward_launch<T, N>(g, in, R, pos, w, T_, K, H, out, gw, s)
             : merge_backward_launch<T, 1>(g, in, R, pos, w, T_, K, H, out, gw, s);
}

}  // namespace
}  // namespace moe

extern "C" {
using namespace moe;

moe_status moe_async_sort_experts(const int32_t* d_expert, int32_t T, int32_t K, int32_t E, int32_t* d_offsets,
                                  int32_t* d_pos, int32_t* d_pair, void* stream) {
  if (T < 0 || K < 1 || K > 32 || E < 1 || E > kMaxExperts || (int64_t)T * K > INT32_MAX - 1024) return MOE_ERR_INVALID;
  if (!d_offsets || (T > 0 && (!d_expert || !d_pos || !d_pair))) return MOE_ERR_INVALID;
  // 128 pairs a warp while that needs no more than 256 warps; over 32 of them, eight CTAs
  const long long P = (long long)T * K;
  const int all = (int)std::max<long long>(4, std::min<long long>(32 * kSortCluster, (P + 127) / 128));
  const int ctas = all > 32 ? kSortCluster : 1, warps = (all + ctas - 1) / ctas;
  const int per = (int)(((P + (long long)warps * ctas - 1) / ((long long)warps * ctas) + 31) & ~31LL);
  const size_t smem = (size_t)(warps + 3) * (E + 1) * sizeof(int);
  // the limit belongs to the function, and another thread may launch it with more at any time: one limit for all calls
  if (smem > 48 * 1024 && cudaFuncSetAttribute(sort_experts_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSortSmem) != cudaSuccess)
    return MOE_ERR_CUDA;
  return launch_op(sort_experts_kernel, dim3(ctas), 32 * warps, smem, ctas, stream, d_expert, (int)P, E, per, d_offsets,
                   d_pos, d_pair);
}

moe_status moe_async_sort_rows(int32_t dtype, const void* d_x, int64_t x_stride, const int32_t* d_pos, int32_t T,
                               int32_t K, int32_t H, void* d_rows, int64_t rows_stride, int64_t n_rows, void* stream) {
  if (!valid_rows(dtype, T, K, H, n_rows)) return MOE_ERR_INVALID;
  if (T == 0 || n_rows == 0) return MOE_OK;
  if (!d_x || !d_pos || !d_rows || x_stride < H || rows_stride < H) return MOE_ERR_INVALID;
  return dtype == MOE_BF16
             ? sort_rows_dispatch<__nv_bfloat16>(d_x, x_stride, d_pos, T, K, H, n_rows, d_rows, rows_stride, stream)
             : sort_rows_dispatch<float>(d_x, x_stride, d_pos, T, K, H, n_rows, d_rows, rows_stride, stream);
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
  return dtype == MOE_BF16 ? merge_rows_dispatch<__nv_bfloat16>(d_rows, rows_stride, n_rows, d_pos, d_w, T, K, H,
                                                              d_residual, residual_stride, d_y, y_stride, stream)
                           : merge_rows_dispatch<float>(d_rows, rows_stride, n_rows, d_pos, d_w, T, K, H, d_residual,
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
             ? merge_backward_dispatch<__nv_bfloat16>(d_grad, grad_stride, d_rows, rows_stride, n_rows, d_pos, d_w, T, K,
                                                    H, d_grad_rows, grad_rows_stride, d_grad_w, stream)
             : merge_backward_dispatch<float>(d_grad, grad_stride, d_rows, rows_stride, n_rows, d_pos, d_w, T, K, H,
                                            d_grad_rows, grad_rows_stride, d_grad_w, stream);
}

moe_status moe_async_route_backward(const int32_t* d_idx, const float* d_w, const float* d_grad_w, int32_t T, int32_t E,
                                    int32_t K, float* d_grad_logits, void* stream) {
  if (T < 0 || E < 1 || E > kMaxExperts || K < 1 || K > E || K > 32) return MOE_ERR_INVALID;
  if (T == 0) return MOE_OK;
  if (!d_idx || !d_w || !d_grad_w || !d_grad_logits) return MOE_ERR_INVALID;
  return launch_op(route_backward_kernel, dim3((unsigned)((T + 7LL) / 8)), 256, 0, 1, stream, d_idx, d_w, d_grad_w, T, E, K,
                   d_grad_logits);
}

}  // extern "C"
