// wfst_lowrank.cu — low-rank adapters of many requests beside a shared
// projection: first form, one CTA per row.
#include "wfst_ops.h"

namespace wfst {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRank = 128;

struct Args {
  const void *y, *x, *shrink, *expand;
  const int32_t* adapter;
  const float* scales;
  void* out;
  int64_t sy, sx, so, ss_a, ss_j, se_a, se_n;
  int32_t rows, n, k, rank, adapters;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) lowrank_kernel(const Args a) {
  __shared__ float t[kMaxRank];
  const int r = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ops_begin();
  ops_next();
  const int which = ops_load(a.adapter + r);
  const bool some = (uint32_t)which < (uint32_t)a.adapters;
  if (some) {
    const T* x = reinterpret_cast<const T*>(a.x) + r * a.sx;
    for (int j = warp; j < a.rank; j += kThreads / 32) {
      const T* s = reinterpret_cast<const T*>(a.shrink) + which * a.ss_a + j * a.ss_j;
      float v = 0.f;
      for (int k = lane; k < a.k; k += 32) v += to_f32(x[k]) * to_f32(s[k]);
      for (int i = 16; i; i /= 2) v += __shfl_xor_sync(0xffffffffu, v, i);
      if (lane == 0) t[j] = v * (a.scales ? a.scales[which] : 1.f);
    }
  }
  __syncthreads();
  for (int n = threadIdx.x; n < a.n; n += kThreads) {
    T v = reinterpret_cast<const T*>(a.y)[r * a.sy + n];
    if (some) {
      const T* e = reinterpret_cast<const T*>(a.expand) + which * a.se_a + n * a.se_n;
      float more = 0.f;
      for (int j = 0; j < a.rank; j++) more += t[j] * to_f32(e[j]);
      v = from_f32<T>(to_f32(v) + more);
    }
    reinterpret_cast<T*>(a.out)[r * a.so + n] = v;
  }
}

}  // namespace
}  // namespace wfst

using namespace wfst;

extern "C" int wfst_add_lowrank(const wfst_lowrank_args* r, void* stream) {
  if (!r) return api_fail(WFST_ERR_INVALID_ARG, "add_lowrank: NULL argument");
  if (r->dtype != WFST_F16 && r->dtype != WFST_BF16) return api_fail(WFST_ERR_INVALID_ARG, "add_lowrank: bad dtype");
  if (r->rows < 0 || r->n < 0 || r->adapters < 0) return api_fail(WFST_ERR_INVALID_ARG, "add_lowrank: counts must be >= 0");
  if (r->k < 8 || r->k % 8 || r->k > INT32_MAX - 4096)
    return api_fail(WFST_ERR_INVALID_ARG, "add_lowrank: k must be a positive multiple of 8");
  if (r->rank < 8 || r->rank % 8 || r->rank > kMaxRank)
    return api_fail(WFST_ERR_INVALID_ARG, "add_lowrank: rank must be a multiple of 8 up to 128");
  if (r->n > INT32_MAX - 4096) return api_fail(WFST_ERR_INVALID_ARG, "add_lowrank: n is too large");
  if (r->rows == 0 || r->n == 0) return WFST_OK;
  if (!r->y || !r->x || !r->adapter || !r->out || (r->adapters && (!r->shrink || !r->expand)))
    return api_fail(WFST_ERR_INVALID_ARG, "add_lowrank: NULL argument");
  for (const void* p : {r->x, r->shrink, r->expand})
    if (!aligned(p, 16)) return api_fail(WFST_ERR_INVALID_ARG, "add_lowrank: x, shrink and expand must be 16-byte aligned");
  auto stride = [&](int64_t s, int64_t n) { return n > 1 ? s : 0; };
  Args a;
  a.sy = stride(r->y_stride, r->rows), a.sx = stride(r->x_stride, r->rows), a.so = stride(r->out_stride, r->rows);
  a.ss_a = stride(r->shrink_stride[0], r->adapters), a.ss_j = r->shrink_stride[1];
  a.se_a = stride(r->expand_stride[0], r->adapters), a.se_n = stride(r->expand_stride[1], r->n);
  if ((a.sx | a.ss_a | a.ss_j | a.se_a | a.se_n) & 7)
    return api_fail(WFST_ERR_INVALID_ARG, "add_lowrank: strides of x, shrink and expand must be multiples of 8 elements");
  const int dev = ops_device(r->device, {r->y, r->x, r->shrink, r->expand, r->adapter, r->scales, r->out});
  if (dev < 0) return api_fail(WFST_ERR_INVALID_ARG, "add_lowrank: every array must be device memory of one device");
  OpsDevice guard(dev);
  if (guard.err != cudaSuccess) return api_cuda_fail(guard.err, "add_lowrank: device");
  a.y = r->y, a.x = r->x, a.shrink = r->shrink, a.expand = r->expand, a.adapter = r->adapter, a.scales = r->scales;
  a.out = r->out, a.rows = r->rows, a.n = r->n, a.k = r->k, a.rank = r->rank, a.adapters = r->adapters;
  auto* fn = r->dtype == WFST_F16 ? lowrank_kernel<__half> : lowrank_kernel<__nv_bfloat16>;
  const cudaError_t e = ops_launch(fn, dim3(a.rows), kThreads, 0, 0, (cudaStream_t)stream, a);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "add_lowrank launch");
}
