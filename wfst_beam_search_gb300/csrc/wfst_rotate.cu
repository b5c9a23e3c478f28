// wfst_rotate.cu — the heads' norm and rotation of a new token, and its write
// into the paged cache, in one pass.
//
//   h' = h / sqrt(mean(h^2) + eps) * gain          (each head of q and of k)
//   the first `rot` elements of h' are turned by the token's position, pairs
//   (i, i + rot/2) or (2i, 2i + 1):  (a, b) -> (a cos - b sin, a sin + b cos)
//   q' is written to q_out; k' and v go to the cache row of the token's slot.
//
// A pass reads q, k and v once and writes them once, so HBM bounds it.  A head
// of D elements is held by D / 8 lanes, 16 bytes each: the norm is a sum over
// those lanes, and a pair's other half is in the same lane or one shuffle
// away.  Everything between the load and the store is fp32, rounded once.
#include "wfst_ops.h"

namespace wfst {
namespace {

constexpr int kThreads = 256;

struct Args {
  const void *q, *k, *v, *qw, *kw;
  const int32_t *pos, *slots;
  const float* table;
  void *qo, *kc, *vc;
  int64_t sq_t, sq_h, sk_t, sk_h, sv_t, sv_h, so_t, so_h;
  int64_t ck_p, ck_s, ck_h, cv_p, cv_s, cv_h;
  int64_t items, capacity;
  int32_t tokens, hq, hkv, rot, page, contexts, inter;
  float eps;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const Args a) {
  constexpr int L = D / 8;  // lanes of one head
  const int lane = threadIdx.x & 31, sub = lane % L, lead = lane - sub;
  const int heads = a.hq + 2 * a.hkv;
  const int64_t step = (int64_t)gridDim.x * (kThreads / L);
  const int64_t first = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / L;
  // whole warps stay in the loop: its shuffles want every lane
  const int64_t rounds = (a.items - ((int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31)) / L + step - 1) / step;
  for (int64_t i = 0; i < rounds; i++) {
    const int64_t item = first + i * step;
    const bool live = item < a.items;
    const int tok = live ? (int)(item / heads) : 0;
    const int head = live ? (int)(item - (int64_t)tok * heads) : 0;
    const bool is_q = head < a.hq, is_k = !is_q && head < a.hq + a.hkv;
    const int h = is_q ? head : is_k ? head - a.hq : head - a.hq - a.hkv;
    const T* src = is_q ? reinterpret_cast<const T*>(a.q) + tok * a.sq_t + h * a.sq_h
                 : is_k ? reinterpret_cast<const T*>(a.k) + tok * a.sk_t + h * a.sk_h
                        : reinterpret_cast<const T*>(a.v) + tok * a.sv_t + h * a.sv_h;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live) raw = *reinterpret_cast<const uint4*>(src + sub * 8);
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const float2 f = unpack2<T>(reinterpret_cast<const uint32_t*>(&raw)[j]);
      x[2 * j] = f.x;
      x[2 * j + 1] = f.y;
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j++) ss += x[j] * x[j];
#pragma unroll
    for (int m = 1; m < L; m *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const bool turn = live && (is_q || is_k);
    const float inv = rsqrtf(ss * (1.f / D) + a.eps);
    const T* gain = reinterpret_cast<const T*>(is_q ? a.qw : a.kw);
    uint4 graw = make_uint4(0, 0, 0, 0);
    if (turn && gain) graw = __ldg(reinterpret_cast<const uint4*>(gain + sub * 8));
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const float2 f = gain ? unpack2<T>(reinterpret_cast<const uint32_t*>(&graw)[j]) : make_float2(1.f, 1.f);
      x[2 * j] *= inv * f.x;
      x[2 * j + 1] *= inv * f.y;
    }
    // the pair's other half: in the same lane, or rot / 16 lanes away
    const int half = a.rot / 2, away = a.rot / 16;
    const bool low = sub < away, turned = sub * 8 < a.rot;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const int from = turned ? lead + (low ? sub + away : sub - away) : lane;
      y[j] = __shfl_sync(0xffffffffu, x[j], from);
    }
    if (a.inter) {
#pragma unroll
      for (int j = 0; j < 8; j++) y[j] = x[j ^ 1];
    }
    if (turn && turned) {
      const int32_t p = a.pos[tok];
      float c[8], s[8];
      if (p >= 0 && p < a.contexts) {
        const float* row = a.table + (int64_t)p * a.rot;
        if (a.inter) {
#pragma unroll
          for (int j = 0; j < 4; j++) {
            c[2 * j] = c[2 * j + 1] = __ldg(row + sub * 4 + j);
            s[2 * j + 1] = __ldg(row + half + sub * 4 + j);
            s[2 * j] = -s[2 * j + 1];
          }
        } else {
          const int at = (low ? sub : sub - away) * 8;
#pragma unroll
          for (int j = 0; j < 8; j++) {
            c[j] = __ldg(row + at + j);
            const float v = __ldg(row + half + at + j);
            s[j] = low ? -v : v;
          }
        }
      } else {  // no such row: the result says so
#pragma unroll
        for (int j = 0; j < 8; j++) c[j] = s[j] = __int_as_float(0x7fffffff);
      }
#pragma unroll
      for (int j = 0; j < 8; j++) x[j] = x[j] * c[j] + y[j] * s[j];
    }
    if (!live) continue;
    uint4 out = raw;
    if (turn) {
#pragma unroll
      for (int j = 0; j < 4; j++) reinterpret_cast<uint32_t*>(&out)[j] = pack2<T>(x[2 * j], x[2 * j + 1]);
    }
    if (is_q) {
      *reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.qo) + tok * a.so_t + h * a.so_h + sub * 8) = out;
    } else {
      const int64_t slot = a.slots[tok];
      if (slot < 0 || slot >= a.capacity) continue;  // a token that is not kept
      const int64_t pg = slot / a.page, off = slot - pg * a.page;
      T* dst = is_k ? reinterpret_cast<T*>(a.kc) + pg * a.ck_p + off * a.ck_s + h * a.ck_h
                    : reinterpret_cast<T*>(a.vc) + pg * a.cv_p + off * a.cv_s + h * a.cv_h;
      *reinterpret_cast<uint4*>(dst + sub * 8) = out;
    }
  }
}

template <typename T, int D>
cudaError_t launch(const Args& a, cudaStream_t st) {
  const int64_t want = (a.items * (D / 8) + kThreads - 1) / kThreads;
  const int64_t most = (int64_t)ops_sm_count() * 8;
  rotate_kernel<T, D><<<(int)(want < most ? want : most), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t by_width(const Args& a, int d, cudaStream_t st) {
  if (d == 64) return launch<T, 64>(a, st);
  if (d == 128) return launch<T, 128>(a, st);
  return launch<T, 256>(a, st);
}

}  // namespace
}  // namespace wfst

using namespace wfst;

extern "C" int wfst_norm_rotate(const wfst_rotate_args* r, void* stream) {
  if (!r) return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: NULL argument");
  if (r->tokens < 0 || r->q_heads < 0 || r->kv_heads < 0)
    return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: counts must be >= 0");
  if (r->dtype != WFST_F16 && r->dtype != WFST_BF16) return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: bad dtype");
  if (r->head_dim != 64 && r->head_dim != 128 && r->head_dim != 256)
    return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: head_dim must be 64, 128 or 256");
  if (r->rot < 0 || r->rot > r->head_dim || r->rot % 16)
    return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: rot must be a multiple of 16 up to head_dim");
  if (!(r->eps >= 0.f)) return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: eps must be >= 0");
  const int64_t heads = (int64_t)r->q_heads + 2 * (int64_t)r->kv_heads;
  if (r->tokens == 0 || heads == 0) return WFST_OK;
  if (heads > INT32_MAX) return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: too many heads");
  if ((r->q_heads && (!r->q || !r->q_out)) || (r->rot && (!r->positions || !r->table)) ||
      (r->kv_heads && (!r->k || !r->v || !r->k_pages || !r->v_pages || !r->slots)))
    return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: NULL argument");
  if (r->kv_heads && (r->page_size < 1 || r->num_pages < 0))
    return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: page_size must be >= 1 and num_pages >= 0");
  if (r->rot && r->contexts < 0) return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: contexts must be >= 0");
  for (const void* p : {r->q, r->k, r->v, r->q_gain, r->k_gain, (const void*)r->q_out, (const void*)r->k_pages,
                        (const void*)r->v_pages})
    if (!aligned(p, 16)) return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: arrays must be 16-byte aligned");
  auto stride = [&](int64_t s, int64_t n) { return n > 1 ? s : 0; };
  Args a;
  a.sq_t = stride(r->q_stride[0], r->tokens), a.sq_h = stride(r->q_stride[1], r->q_heads);
  a.sk_t = stride(r->k_stride[0], r->tokens), a.sk_h = stride(r->k_stride[1], r->kv_heads);
  a.sv_t = stride(r->v_stride[0], r->tokens), a.sv_h = stride(r->v_stride[1], r->kv_heads);
  a.so_t = stride(r->out_stride[0], r->tokens), a.so_h = stride(r->out_stride[1], r->q_heads);
  a.ck_p = stride(r->k_page_stride[0], r->num_pages), a.ck_s = stride(r->k_page_stride[1], r->page_size);
  a.cv_p = stride(r->v_page_stride[0], r->num_pages), a.cv_s = stride(r->v_page_stride[1], r->page_size);
  a.ck_h = stride(r->k_page_stride[2], r->kv_heads), a.cv_h = stride(r->v_page_stride[2], r->kv_heads);
  if ((a.sq_t | a.sq_h | a.sk_t | a.sk_h | a.sv_t | a.sv_h | a.so_t | a.so_h | a.ck_p | a.ck_s | a.ck_h | a.cv_p |
       a.cv_s | a.cv_h) & 7)
    return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: strides must be multiples of 8 elements");
  const int dev = ops_device(r->device, {r->q, r->k, r->v, r->q_gain, r->k_gain, r->positions, r->slots, r->table, r->q_out,
                              r->k_pages, r->v_pages});
  if (dev < 0) return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: every array must be device memory of one device");
  OpsDevice guard(dev);
  if (guard.err != cudaSuccess) return api_cuda_fail(guard.err, "norm_rotate: device");
  a.q = r->q, a.k = r->k, a.v = r->v, a.qw = r->q_gain, a.kw = r->k_gain;
  a.pos = r->positions, a.slots = r->slots, a.table = r->table;
  a.qo = r->q_out, a.kc = r->k_pages, a.vc = r->v_pages;
  a.items = heads * r->tokens;
  a.capacity = r->kv_heads ? (int64_t)r->num_pages * r->page_size : 0;
  a.tokens = r->tokens, a.hq = r->q_heads, a.hkv = r->kv_heads, a.rot = r->rot;
  a.page = r->page_size, a.contexts = r->contexts, a.inter = r->interleaved != 0;
  a.eps = r->eps;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = r->dtype == WFST_F16 ? by_width<__half>(a, r->head_dim, st)
                                             : by_width<__nv_bfloat16>(a, r->head_dim, st);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "norm_rotate launch");
}
