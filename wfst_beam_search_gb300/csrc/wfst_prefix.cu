// wfst_prefix.cu — attention of one new token per lane behind a prefix that all
// lanes share: first form, one CTA per lane and query head, one key to a warp at
// a time.
#include "wfst_ops.h"

namespace wfst {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Args {
  const void *q, *kc, *vc;
  const int32_t *shared, *shared_len, *table, *lens;
  void* o;
  float* lse;
  int64_t sq_b, sq_h, so_b, so_h, sl_b;
  int64_t ck_p, ck_s, ck_h, cv_p, cv_s, cv_h, st_b;
  int32_t share, shared_width, width, page, num_pages;
  float scale;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) prefix_kernel(const Args a) {
  __shared__ float acc[kWarps][D], ms[kWarps], ls[kWarps];
  const int b = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ops_begin();
  ops_next();
  const int first = (int)max((int64_t)0, min((int64_t)*a.shared_len, (int64_t)a.shared_width * a.page));
  const int mine = (int)max((int64_t)0, min((int64_t)a.lens[b], (int64_t)a.width * a.page));
  float q[D / 32], o[D / 32], m = -INFINITY, l = 0.f;
  for (int i = 0; i < D / 32; i++) {
    q[i] = to_f32(ops_load(reinterpret_cast<const T*>(a.q) + b * a.sq_b + h * a.sq_h + i * 32 + lane)) * a.scale;
    o[i] = 0.f;
  }
  for (int64_t j = warp; j < (int64_t)first + mine; j += kWarps) {
    const int64_t key = j < first ? j : j - first;
    const int32_t page = ops_load(j < first ? a.shared + key / a.page : a.table + b * a.st_b + key / a.page);
    if ((uint32_t)page >= (uint32_t)a.num_pages) continue;
    const T* k = reinterpret_cast<const T*>(a.kc) + page * a.ck_p + key % a.page * a.ck_s + h / a.share * a.ck_h;
    const T* v = reinterpret_cast<const T*>(a.vc) + page * a.cv_p + key % a.page * a.cv_s + h / a.share * a.cv_h;
    float x = 0.f;
    for (int i = 0; i < D / 32; i++) x += q[i] * to_f32(k[i * 32 + lane]);
    for (int s = 16; s; s /= 2) x += __shfl_xor_sync(0xffffffffu, x, s);
    const float now = fmaxf(m, x), ref = now == -INFINITY ? 0.f : now, keep = expf(m - ref), p = expf(x - ref);
    m = now;
    l = l * keep + p;
    for (int i = 0; i < D / 32; i++) o[i] = o[i] * keep + p * to_f32(v[i * 32 + lane]);
  }
  if (lane == 0) ms[warp] = m, ls[warp] = l;
  for (int i = 0; i < D / 32; i++) acc[warp][i * 32 + lane] = o[i];
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; w++) top = fmaxf(top, ms[w]);
  const float ref = top == -INFINITY ? 0.f : top;
  for (int w = 0; w < kWarps; w++) sum += ls[w] * expf(ms[w] - ref);
  for (int i = threadIdx.x; i < D; i += kThreads) {
    float v = 0.f;
    for (int w = 0; w < kWarps; w++) v += acc[w][i] * expf(ms[w] - ref);
    reinterpret_cast<T*>(a.o)[b * a.so_b + h * a.so_h + i] = from_f32<T>(sum == 0.f ? 0.f : v / sum);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[b * a.sl_b + h] = top + logf(sum);
}

template <typename T>
cudaError_t launch(const Args& a, int d, int lanes, int heads, cudaStream_t st) {
  auto* fn = d == 64 ? prefix_kernel<T, 64> : d == 128 ? prefix_kernel<T, 128> : prefix_kernel<T, 256>;
  return ops_launch(fn, dim3(lanes, heads), kThreads, 0, 0, st, a);
}

}  // namespace
}  // namespace wfst

using namespace wfst;

extern "C" int wfst_prefix_size(int32_t lanes, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t* bytes) {
  if (!bytes) return api_fail(WFST_ERR_INVALID_ARG, "prefix_size: NULL argument");
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return api_fail(WFST_ERR_INVALID_ARG, "prefix_size: head_dim must be 64, 128 or 256");
  if (lanes < 0 || q_heads < 0) return api_fail(WFST_ERR_INVALID_ARG, "prefix_size: counts must be >= 0");
  if (kv_heads < 1 || q_heads % kv_heads)
    return api_fail(WFST_ERR_INVALID_ARG, "prefix_size: q_heads must be a multiple of kv_heads");
  if ((int64_t)lanes * q_heads > INT32_MAX) return api_fail(WFST_ERR_INVALID_ARG, "prefix_size: too many heads");
  return wfst_attend_size(bytes);
}

extern "C" int wfst_attend_prefix(const wfst_prefix_args* r, void* stream) {
  if (!r) return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: NULL argument");
  if (r->dtype != WFST_F16 && r->dtype != WFST_BF16) return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: bad dtype");
  int64_t bytes;
  if (const int rc = wfst_prefix_size(r->lanes, r->q_heads, r->kv_heads, r->head_dim, &bytes)) return rc;
  if (r->page_size < 1 || r->num_pages < 0 || r->table_width < 0 || r->prefix_width < 0)
    return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: page_size must be >= 1, num_pages and table widths >= 0");
  if ((int64_t)r->page_size * r->table_width > INT32_MAX - 1024 || (int64_t)r->page_size * r->prefix_width > INT32_MAX - 1024)
    return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: page_size times a table's width must stay below 2^31");
  if (!(r->scale == r->scale)) return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: scale must be a number");
  if (r->lanes == 0 || r->q_heads == 0) return WFST_OK;
  if (!r->q || !r->o || !r->prefix_length || !r->lengths || !r->workspace || (r->prefix_width && !r->prefix_table) ||
      (r->table_width && !r->table) || (r->num_pages && (!r->k_pages || !r->v_pages)))
    return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: NULL argument");
  for (const void* p : {r->q, r->k_pages, r->v_pages, (const void*)r->workspace})
    if (!aligned(p, 16)) return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: arrays must be 16-byte aligned");
  auto stride = [&](int64_t s, int64_t n) { return n > 1 ? s : 0; };
  Args a;
  a.sq_b = stride(r->q_stride[0], r->lanes), a.sq_h = stride(r->q_stride[1], r->q_heads);
  a.ck_p = stride(r->k_page_stride[0], r->num_pages), a.ck_s = stride(r->k_page_stride[1], r->page_size);
  a.cv_p = stride(r->v_page_stride[0], r->num_pages), a.cv_s = stride(r->v_page_stride[1], r->page_size);
  a.ck_h = stride(r->k_page_stride[2], r->kv_heads), a.cv_h = stride(r->v_page_stride[2], r->kv_heads);
  if ((a.sq_b | a.sq_h | a.ck_p | a.ck_s | a.ck_h | a.cv_p | a.cv_s | a.cv_h) & 7)
    return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: strides must be multiples of 8 elements");
  const int dev = ops_device(r->device, {r->q, r->k_pages, r->v_pages, r->prefix_table, r->prefix_length, r->table, r->lengths,
                                         r->o, r->lse, r->workspace});
  if (dev < 0) return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: every array must be device memory of one device");
  OpsDevice guard(dev);
  if (guard.err != cudaSuccess) return api_cuda_fail(guard.err, "attend_prefix: device");
  a.q = r->q, a.kc = r->k_pages, a.vc = r->v_pages;
  a.shared = r->prefix_table, a.shared_len = r->prefix_length, a.table = r->table, a.lens = r->lengths;
  a.o = r->o, a.lse = r->lse;
  a.so_b = stride(r->o_stride[0], r->lanes), a.so_h = stride(r->o_stride[1], r->q_heads), a.sl_b = r->lse_stride;
  a.st_b = stride(r->table_stride, r->lanes);
  a.share = r->q_heads / r->kv_heads, a.shared_width = r->prefix_width, a.width = r->table_width;
  a.page = r->page_size, a.num_pages = r->num_pages, a.scale = r->scale;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = r->dtype == WFST_F16 ? launch<__half>(a, r->head_dim, r->lanes, r->q_heads, st)
                                             : launch<__nv_bfloat16>(a, r->head_dim, r->lanes, r->q_heads, st);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "attend_prefix launch");
}
