// wfst_ops.h — what the second-pass operators share: element types, argument
// checks, launches on the tensors' own device.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "../../include/wfst_gb300.h"

namespace wfst {

int api_fail(int code, const char* msg);
int api_cuda_fail(cudaError_t e, const char* what);

// Every array of these calls is device memory of one device: `given` where the
// caller knows it.  Otherwise asks the driver; -1 when a pointer is not device
// memory or lies elsewhere; NULL entries (optional arrays) are skipped.
inline int ops_device(int given, std::initializer_list<const void*> ptrs) {
  if (given >= 0) return given;
  int dev = -1;
  for (const void* p : ptrs) {
    if (!p) continue;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
      cudaGetLastError();
      return -1;
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) return -1;
    if (dev >= 0 && at.device != dev) return -1;
    dev = at.device;
  }
  return dev;
}

// Makes `dev` current for a launch and puts the caller's device back.
struct OpsDevice {
  int prev = -1, dev;
  cudaError_t err;
  explicit OpsDevice(int d) : dev(d) {
    err = cudaGetDevice(&prev);
    if (err == cudaSuccess && prev != dev) err = cudaSetDevice(dev);
    if (err != cudaSuccess) cudaGetLastError();
  }
  ~OpsDevice() {
    if (prev >= 0 && prev != dev) cudaSetDevice(prev);
  }
  OpsDevice(const OpsDevice&) = delete;
};

// What a kernel needs set up once per device (its shared memory size): the
// flags of the devices where that is done.
struct OpsOnce {
  std::atomic<uint64_t> done{0};
  bool operator()(int dev) const { return dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1); }
  void set(int dev) { done.fetch_or(dev < 64 ? (uint64_t)1 << dev : 0, std::memory_order_release); }
};

// Multiprocessors of the current device (cached per device; 152 on GB300).
int ops_sm_count();
inline int ops_current() {
  int d = 0;
  cudaGetDevice(&d);
  return d;
}

// wfst_attend_paged of checked arguments.  With `own` m, l and o are left there
// unscaled, as the attention kernels hold them (m [rows], l [rows], o
// [rows][head_dim]; rows: lanes * q_heads up to a multiple of 4, by key-value head,
// lane, head of it), and o and lse are not written; the kernel then starts while the one before it in
// the stream, which has to be ops_launch's, still runs, and ends after it.
int attend_behind(const wfst_attend_args* args, float* own, void* stream);

#ifdef __CUDACC__

// Launches `fn` so that its CTAs may be set up while the kernel before it in the
// stream ends (a step is a chain of short kernels).  Every kernel launched like
// this calls ops_begin in all its threads before it touches memory that any
// kernel writes, and before it takes tensor memory; ops_next, after that, lets
// the one behind it set up.
template <typename... P>
cudaError_t ops_launch(void (*fn)(P...), dim3 grid, int threads, int smem, int cluster, cudaStream_t st,
                       const std::common_type_t<P>&... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = cluster ? 2 : 1;  // 0: a kernel that knows no clusters
  return cudaLaunchKernelEx(&cfg, fn, args...);
}
__device__ __forceinline__ void ops_begin() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Loads that the compiler keeps behind ops_begin, as it need not keep those of
// the read-only path; the second one's data are not read again.
template <typename V>
__device__ __forceinline__ V ops_load(const V* p) {
  return *p;
}
__device__ __forceinline__ uint4 ops_load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void ops_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

#endif

inline bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

#ifdef __CUDACC__

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The two 16-bit values of a 32-bit word, widened.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Two floats rounded to one 32-bit word of 16-bit values (first one low).
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// c += a (16x16) * b (16x8), fp32 accumulation; one warp.
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

#endif  // __CUDACC__
}  // namespace wfst
