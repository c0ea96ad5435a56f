// What the stateless operators (sorted dispatch, norm, product) share: launches, argument
// checks and 16-byte or element-wise access to rows.
#pragma once
#include "moe_internal.cuh"

namespace moe {

// A row is read in units of V elements: 16 bytes where every row starts on a 16-byte boundary
// and holds whole vectors, single elements otherwise.
template <typename T, int V> struct RowVec;
template <typename T> struct RowVec<T, 1> {
  using Raw = T;
  static __device__ __forceinline__ Raw load(const T* p) { return __ldg(p); }
  static __device__ __forceinline__ Raw load_rw(const T* p) { return *p; }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[1]) { v[0] = to_f(r); }
  static __device__ __forceinline__ Raw pack(const float (&v)[1]) { return from_f<T>(v[0]); }
  static __device__ __forceinline__ void store(T* p, const Raw& r) { *p = r; }
};
template <typename T> struct RowVec<T, Vec<T>::N> {
  using Raw = uint4;
  static __device__ __forceinline__ Raw load(const T* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
  static __device__ __forceinline__ Raw load_rw(const T* p) { return *reinterpret_cast<const uint4*>(p); }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&v)[Vec<T>::N]) { unpack16<T>(r, v); }
  static __device__ __forceinline__ Raw pack(const float (&v)[Vec<T>::N]) { return pack16<T>(v); }
  static __device__ __forceinline__ void store(T* p, const Raw& r) { *reinterpret_cast<uint4*>(p) = r; }
};

// Row operand: base and row stride in elements.
template <typename T> struct Rows {
  T* p;
  int64_t ld;
  __device__ __forceinline__ T* at(int64_t r) const { return p + r * ld; }
};

// Column indices are 32-bit and step past a row's end by up to a block's columns (at most 512 x 8 a step, four of them).
constexpr int kMaxWidth = INT32_MAX - 65536;

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// 16-byte access to rows at p with row stride ld (elements of `size` bytes); a null p has no say.
inline bool rows16(const void* p, int64_t ld, int size) { return !p || (aligned16(p) && ld * size % 16 == 0); }

inline int dtype_size(int32_t dtype) { return dtype == MOE_F32 ? 4 : dtype == MOE_BF16 ? 2 : 1; }

// A launch that may start while the kernel before it in the stream still runs: the kernel
// waits (ops_begin) before it touches memory.
__device__ __forceinline__ void ops_begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... KArgs, typename... Args>
moe_status launch_op(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster, void* stream,
                     Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

}  // namespace moe
