// wfst_score.cu — how likely given tokens are: first form, one CTA per row, the
// alternatives one by one.
#include "wfst_ops.h"

namespace wfst {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Args {
  const void* logits;
  const int32_t* tokens;
  float *logprobs, *entropy;
  int32_t* top_tokens;
  float* top_logprobs;
  int64_t stride;
  int32_t rows, vocab, top;
};

// Larger logit, larger key; -0 and +0 have one; then lower index.  0: no logit.
__device__ __forceinline__ uint64_t order_of(float v, int e) {
  if (!(v > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(v + 0.f);
  return (uint64_t)(b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u)) << 32 | (0xffffffffu - (uint32_t)e);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) score_kernel(const Args a) {
  __shared__ float red[3][kWarps];
  __shared__ uint64_t best[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  ops_begin();
  ops_next();
  const T* x = reinterpret_cast<const T*>(a.logits) + blockIdx.x * a.stride;
  float m = -INFINITY;
  for (int i = tid; i < a.vocab; i += kThreads) m = fmaxf(m, to_f32(x[i]));
  for (int s = 16; s; s /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
  for (int w = 0; w < kWarps; w++) m = fmaxf(m, red[0][w]);
  const float ref = m == -INFINITY ? 0.f : m;
  float z = 0.f, u = 0.f;
  for (int i = tid; i < a.vocab; i += kThreads) {
    const float y = to_f32(x[i]) - ref, e = expf(y);
    z += e;
    u += e == 0.f ? 0.f : e * y;
  }
  for (int s = 16; s; s /= 2) z += __shfl_xor_sync(0xffffffffu, z, s), u += __shfl_xor_sync(0xffffffffu, u, s);
  if (lane == 0) red[1][warp] = z, red[2][warp] = u;
  __syncthreads();
  z = u = 0.f;
  for (int w = 0; w < kWarps; w++) z += red[1][w], u += red[2][w];
  const float log_z = logf(z);
  if (tid == 0) {
    const int t = ops_load(a.tokens + blockIdx.x);
    float v = 0.f;
    if (t >= a.vocab)
      v = NAN;
    else if (t >= 0)
      v = z == 0.f ? -INFINITY : to_f32(x[t]) - ref - log_z;
    a.logprobs[blockIdx.x] = v;
    a.entropy[blockIdx.x] = z == 0.f ? 0.f : log_z - u / z;
  }
  uint64_t before = ~(uint64_t)0;
  for (int j = 0; j < a.top; j++) {
    uint64_t next = 0;
    for (int i = tid; i < a.vocab; i += kThreads) {
      const uint64_t o = order_of(to_f32(x[i]), i);
      if (o < before && o > next) next = o;
    }
    for (int s = 16; s; s /= 2) next = max(next, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)next, s));
    __syncthreads();
    if (lane == 0) best[warp] = next;
    __syncthreads();
    for (int w = 0; w < kWarps; w++) next = max(next, best[w]);
    before = next;
    if (tid == 0) {
      const int e = next ? (int)(0xffffffffu - (uint32_t)next) : -1;
      a.top_tokens[(int64_t)blockIdx.x * a.top + j] = e;
      a.top_logprobs[(int64_t)blockIdx.x * a.top + j] = next ? to_f32(x[e]) - ref - log_z : -INFINITY;
    }
  }
}

}  // namespace
}  // namespace wfst

using namespace wfst;

extern "C" int wfst_score_tokens(const wfst_score_args* r, void* stream) {
  if (!r) return api_fail(WFST_ERR_INVALID_ARG, "score_tokens: NULL argument");
  if (r->dtype != WFST_F32 && r->dtype != WFST_F16 && r->dtype != WFST_BF16)
    return api_fail(WFST_ERR_INVALID_ARG, "score_tokens: bad dtype");
  if (r->rows < 0) return api_fail(WFST_ERR_INVALID_ARG, "score_tokens: rows must be >= 0");
  if (r->vocab < 1 || r->vocab > 1 << 20) return api_fail(WFST_ERR_INVALID_ARG, "score_tokens: vocab must be 1 to 2^20");
  if (r->top < 0 || r->top > WFST_SCORE_TOP) return api_fail(WFST_ERR_INVALID_ARG, "score_tokens: top must be 0 to 64");
  if (r->rows > 1 && r->stride < r->vocab) return api_fail(WFST_ERR_INVALID_ARG, "score_tokens: stride must be >= vocab");
  if (r->rows == 0) return WFST_OK;
  if (!r->logits || !r->tokens || !r->logprobs || !r->entropy || (r->top && (!r->top_tokens || !r->top_logprobs)))
    return api_fail(WFST_ERR_INVALID_ARG, "score_tokens: NULL argument");
  const int dev = ops_device(r->device, {r->logits, r->tokens, r->logprobs, r->entropy, r->top ? r->top_tokens : nullptr,
                                         r->top ? r->top_logprobs : nullptr});
  if (dev < 0) return api_fail(WFST_ERR_INVALID_ARG, "score_tokens: every array must be device memory of one device");
  OpsDevice guard(dev);
  if (guard.err != cudaSuccess) return api_cuda_fail(guard.err, "score_tokens: device");
  const Args a = {r->logits, r->tokens, r->logprobs, r->entropy, r->top_tokens, r->top_logprobs,
                  r->rows > 1 ? r->stride : 0, r->rows, r->vocab, r->top};
  auto* fn = r->dtype == WFST_F32 ? score_kernel<float> : r->dtype == WFST_F16 ? score_kernel<__half> : score_kernel<__nv_bfloat16>;
  const cudaError_t e = ops_launch(fn, dim3(a.rows), kThreads, 0, 0, (cudaStream_t)stream, a);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "score_tokens launch");
}
