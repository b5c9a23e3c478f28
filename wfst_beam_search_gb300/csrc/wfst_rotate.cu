// wfst_rotate.cu — the heads' norm and rotation of a new token, and its write
// into the paged cache, in one pass.
//
//   h' = h / sqrt(mean(h^2) + eps) * gain          (each head of q and of k)
//   the first `rot` elements of h' are turned by the token's position, pairs
//   (i, i + rot/2) or (2i, 2i + 1):  (a, b) -> (a cos - b sin, a sin + b cos)
//   q' is written to q_out; k' and v go to the cache row of the token's slot.
//
// A pass reads q, k and v once and writes them once, so HBM bounds it, if the
// arithmetic stays small beside it and enough loads are in flight.  A chunk is
// 2 KB of one token's heads, in the order q, k, v; a warp takes a run of
// chunks and copies them ahead of its work, with the token's row of the table,
// into its own ring in shared memory.  A head of D elements is then held by D /
// 8 lanes, four elements from either half of the pairs each: the norm is a sum
// over those lanes, a pair lies within a lane, and gain and turn are one
// product with four factors per pair that a lane keeps for all its heads of a
// kind.  Everything between the load and the store is fp32, rounded once.
//
// 16000 tokens of 32 + 8 + 8 heads of 128 (393 MB) take 65 us, 6.0 TB/s, nine
// tenths of a plain copy's rate; without the copies ahead, loads straight to
// registers, it was 147.  What is left is the pace of the instructions beside
// the copies (half of the issue slots).  One token takes 2.3 us, a launch.
#include "wfst_ops.h"

namespace wfst {
namespace {

constexpr int kWarps = 8;
constexpr int kStages = 2;       // of a warp's ring: 16000 tokens 66 us, with three 72
constexpr int kChunk = 2048;     // bytes of heads
constexpr int kPasses = kChunk / 512;
template <int D>
constexpr int kStage = kChunk + D * 4;  // with a row of the table behind

struct Args {
  const void *q, *k, *v, *qw, *kw;
  const int32_t *pos, *slots;
  const float* table;
  void *qo, *kc, *vc;
  int64_t sq_t, sq_h, sk_t, sk_h, sv_t, sv_h, so_t, so_h;
  int64_t ck_p, ck_s, ck_h, cv_p, cv_s, cv_h;
  int64_t capacity;
  int64_t items;
  int32_t tokens, hq, hkv, rot, page, contexts, inter, chunks;
  float eps;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Two fp32 values in one 64-bit register, and products on both at once.
__device__ __forceinline__ uint64_t both(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 each(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float rsqrta(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// FULL: the whole head is turned.
template <typename T, int D, bool INTER, bool FULL>
__global__ void __launch_bounds__(kWarps * 32, 2) rotate_kernel(const Args a) {
  constexpr int L = D / 8;                  // lanes of one head
  constexpr int H = kChunk / (2 * D);       // heads of a chunk
  constexpr int R = 32 / L;                 // heads of a pass
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % L, line = lane / L;
  const int heads = a.hq + 2 * a.hkv, turns = a.hq + a.hkv, half = a.rot / 2;
  // neighbouring runs of chunks go to different CTAs, so that few of them spread
  const int64_t w = blockIdx.x + (int64_t)warp * gridDim.x, W = (int64_t)gridDim.x * kWarps;
  const int64_t i0 = a.items * w / W, i1 = a.items * (w + 1) / W;
  ops_begin();
  ops_next();
  if (i0 >= i1) return;
  unsigned char* ring = smem + warp * (kStages * kStage<D>);
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);

  // the lane's elements: [lo, lo + 4) and [hi, hi + 4); pairs are (lo + j, hi
  // + j), or neighbours within either when interleaved
  const bool turned = FULL || sub * 8 < a.rot;
  const int lo = !INTER && turned ? sub * 4 : sub * 8, hi = !INTER && turned ? lo + half : lo + 4;

  // ---- copying ahead: chunk `c_ahead` of token `t_ahead` next
  int t_ahead = (int)(i0 / a.chunks), c_ahead = (int)(i0 - (int64_t)t_ahead * a.chunks);
  int64_t left = i1 - i0;
  int put = 0;
  bool row_due = true;  // the token's row of the table is not in the ring yet
  int32_t pos = a.rot ? ops_load(a.pos + t_ahead) : 0;
  auto copy_next = [&]() {
    if (left > 0) {
      const uint32_t dst = ring_at + put * kStage<D> + lane * 16;
      const int c0 = c_ahead * H;
      const T* src;
      int64_t step;
      if (c0 + H <= a.hq || (c0 >= a.hq && c0 + H <= turns) || (c0 >= turns && c0 + H <= heads)) {
        // heads of one kind
        if (c0 < a.hq) {
          src = reinterpret_cast<const T*>(a.q) + t_ahead * a.sq_t + c0 * a.sq_h, step = a.sq_h;
        } else if (c0 < turns) {
          src = reinterpret_cast<const T*>(a.k) + t_ahead * a.sk_t + (c0 - a.hq) * a.sk_h, step = a.sk_h;
        } else {
          src = reinterpret_cast<const T*>(a.v) + t_ahead * a.sv_t + (c0 - turns) * a.sv_h, step = a.sv_h;
        }
        src += line * step + sub * 8;
#pragma unroll
        for (int i = 0; i < kPasses; i++) copy16(dst + i * 512, src + i * (R * step));
      } else {
#pragma unroll 1
        for (int i = 0; i < kPasses; i++) {
          const int h = c0 + i * R + line;
          if (h >= heads) break;
          src = h < a.hq    ? reinterpret_cast<const T*>(a.q) + t_ahead * a.sq_t + h * a.sq_h
                : h < turns ? reinterpret_cast<const T*>(a.k) + t_ahead * a.sk_t + (h - a.hq) * a.sk_h
                            : reinterpret_cast<const T*>(a.v) + t_ahead * a.sv_t + (h - turns) * a.sv_h;
          copy16(dst + i * 512, src + sub * 8);
        }
      }
      if (row_due && a.rot && pos >= 0 && pos < a.contexts) {
        const float* row = a.table + (int64_t)pos * a.rot + lane * 4;
        for (int i = lane * 4; i < a.rot; i += 128, row += 128) copy16(dst + kChunk + (i - lane * 4) * 4, row);
      }
      left--;
      row_due = false;
      if (++c_ahead == a.chunks) {
        c_ahead = 0;
        t_ahead++;
        row_due = true;
        if (left > 0 && a.rot) pos = ops_load(a.pos + t_ahead);
      }
      put = put + 1 == kStages ? 0 : put + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; i++) copy_next();

  // the gains of this lane's elements
  uint2 gq[2], gk[2];
  auto gain_of = [&](uint2 (&g)[2], const void* w) {
    const T* p = reinterpret_cast<const T*>(w);
    const uint32_t one = pack2<T>(1.f, 1.f);
    g[0] = p ? ops_load(reinterpret_cast<const uint2*>(p + lo)) : make_uint2(one, one);
    g[1] = p ? ops_load(reinterpret_cast<const uint2*>(p + hi)) : make_uint2(one, one);
  };
  gain_of(gq, a.qw);
  gain_of(gk, a.kw);

  // A lane's eight elements are four words of two.  A word turns into (itself *
  // keep + its partner * add), the partner being the word of the pairs' other
  // half, or, interleaved, itself with its two values exchanged; gain and turn
  // are in the factors.
  float c[4], s[4];  // of the lane's four pairs
  uint64_t keep[4], add[4];
  auto factors = [&](const uint2 (&r)[2]) {
    const float2 g0 = unpack2<T>(r[0].x), g1 = unpack2<T>(r[0].y), g2 = unpack2<T>(r[1].x), g3 = unpack2<T>(r[1].y);
    if (INTER) {
      const float2 g[4] = {g0, g1, g2, g3};
#pragma unroll
      for (int v = 0; v < 4; v++) {
        keep[v] = both(g[v].x * c[v], g[v].y * c[v]);
        add[v] = both(-g[v].y * s[v], g[v].x * s[v]);
      }
    } else {
      keep[0] = both(g0.x * c[0], g0.y * c[1]), keep[1] = both(g1.x * c[2], g1.y * c[3]);
      keep[2] = both(g2.x * c[0], g2.y * c[1]), keep[3] = both(g3.x * c[2], g3.y * c[3]);
      add[0] = both(-g2.x * s[0], -g2.y * s[1]), add[1] = both(-g3.x * s[2], -g3.y * s[3]);
      add[2] = both(g0.x * s[0], g0.y * s[1]), add[3] = both(g1.x * s[2], g1.y * s[3]);
    }
  };

  int tok = (int)(i0 / a.chunks), chunk = (int)(i0 - (int64_t)tok * a.chunks);
  bool fresh = true, of_k = false;
  T *q_to = nullptr, *k_to = nullptr, *v_to = nullptr;  // the token's q_out, its cache row
  bool kept = false;
  int get = 0;
  for (int64_t i = i0; i < i1; i++) {
    int32_t slot = -1, p = 0;
    if (fresh) {
      if (a.slots) slot = ops_load(a.slots + tok);
      if (a.rot) p = ops_load(a.pos + tok);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
    copy_next();
    const unsigned char* stage = ring + get * kStage<D>;
    get = get + 1 == kStages ? 0 : get + 1;
    if (fresh) {  // a new token: its turn and its cache row
      const bool known = p >= 0 && p < a.contexts;
      const float* row = reinterpret_cast<const float*>(stage + kChunk) + sub * 4;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        c[j] = 1.f, s[j] = 0.f;
        if (turned && a.rot) {  // a position without a row: the result says so
          c[j] = known ? row[j] : __int_as_float(0x7fffffff);
          s[j] = known ? row[half + j] : __int_as_float(0x7fffffff);
        }
      }
      kept = slot >= 0 && slot < a.capacity;
      const int64_t pg = kept ? slot / a.page : 0, off = kept ? slot - (int32_t)pg * a.page : 0;
      q_to = reinterpret_cast<T*>(a.qo) + tok * a.so_t;
      k_to = reinterpret_cast<T*>(a.kc) + pg * a.ck_p + off * a.ck_s;
      v_to = reinterpret_cast<T*>(a.vc) + pg * a.cv_p + off * a.cv_s;
    }
    const int c0 = chunk * H, h0 = c0 + line;
    if (fresh || (!of_k && h0 >= a.hq)) {
      of_k = h0 >= a.hq;
      factors(of_k ? gk : gq);
    }
    fresh = false;

    const T* in = reinterpret_cast<const T*>(stage) + line * D;
    uint2 raw[kPasses][2];
#pragma unroll
    for (int u = 0; u < kPasses; u++) {
      raw[u][0] = *reinterpret_cast<const uint2*>(in + u * (R * D) + lo);
      raw[u][1] = *reinterpret_cast<const uint2*>(in + u * (R * D) + hi);
    }
    uint64_t x[kPasses][4];
    float inv[kPasses];
    if (c0 < turns) {
#pragma unroll
      for (int u = 0; u < kPasses; u++) {
        uint64_t ss = 0;
#pragma unroll
        for (int v = 0; v < 4; v++) {
          const float2 f = unpack2<T>(v & 1 ? raw[u][v >> 1].y : raw[u][v >> 1].x);
          x[u][v] = both(f.x, f.y);
          ss = v ? fma2(x[u][v], x[u][v], ss) : mul2(x[u][v], x[u][v]);
        }
        inv[u] = each(ss).x + each(ss).y;
      }
#pragma unroll
      for (int m = 1; m < L; m *= 2)
#pragma unroll
        for (int u = 0; u < kPasses; u++) inv[u] += __shfl_xor_sync(0xffffffffu, inv[u], m);
#pragma unroll
      for (int u = 0; u < kPasses; u++) inv[u] = rsqrta(inv[u] * (1.f / D) + a.eps);
    }
    auto turn = [&](int u) {
      const uint64_t scale = both(inv[u], inv[u]);
      uint32_t out[4];
#pragma unroll
      for (int v = 0; v < 4; v++) {
        uint64_t y = mul2(x[u][v], keep[v]);
        if (FULL || turned) {
          const float2 o = each(x[u][v]);
          y = fma2(INTER ? both(o.y, o.x) : x[u][v ^ 2], add[v], y);
        }
        const float2 f = each(mul2(y, scale));
        out[v] = pack2<T>(f.x, f.y);
      }
      raw[u][0] = make_uint2(out[0], out[1]);
      raw[u][1] = make_uint2(out[2], out[3]);
    };
    auto store = [&](T* dst, int u) {
      *reinterpret_cast<uint2*>(dst + lo) = raw[u][0];
      *reinterpret_cast<uint2*>(dst + hi) = raw[u][1];
    };
    if (c0 + H <= a.hq || (c0 >= a.hq && c0 + H <= turns) || (c0 >= turns && c0 + H <= heads)) {
      // heads of one kind
      T* dst;
      int64_t step;
      if (c0 < a.hq) {
        dst = q_to + h0 * a.so_h, step = a.so_h;
      } else if (c0 < turns) {
        dst = k_to + (h0 - a.hq) * a.ck_h, step = a.ck_h;
      } else {
        dst = v_to + (h0 - turns) * a.cv_h, step = a.cv_h;
      }
      if (c0 < turns) {
#pragma unroll
        for (int u = 0; u < kPasses; u++) turn(u);
      }
      if (c0 < a.hq || kept) {
#pragma unroll
        for (int u = 0; u < kPasses; u++) store(dst + u * (R * step), u);
      }
    } else {
#pragma unroll
      for (int u = 0; u < kPasses; u++) {
        const int h = h0 + u * R;
        if (h >= heads) continue;
        if (h < turns) {
          if (!of_k && h >= a.hq) {
            of_k = true;
            factors(gk);
          }
          turn(u);
        }
        if (h < a.hq)
          store(q_to + h * a.so_h, u);
        else if (kept)
          store(h < turns ? k_to + (h - a.hq) * a.ck_h : v_to + (h - turns) * a.cv_h, u);
      }
    }
    if (++chunk == a.chunks) {
      chunk = 0;
      tok++;
      fresh = true;
    }
  }
}

template <typename T, int D>
cudaError_t launch(Args& a, cudaStream_t st) {
  constexpr int smem = kWarps * kStages * kStage<D>;
  auto set_up = [](auto* fn) {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  };
  static OpsOnce once;
  if (const int dev = ops_current(); !once(dev)) {
    for (auto* fn : {rotate_kernel<T, D, true, true>, rotate_kernel<T, D, true, false>,
                     rotate_kernel<T, D, false, true>, rotate_kernel<T, D, false, false>})
      if (const cudaError_t e = set_up(fn); e != cudaSuccess) return e;
    once.set(dev);
  }
  a.chunks = ((a.hq + 2 * a.hkv) * 2 * D + kChunk - 1) / kChunk;
  a.items = (int64_t)a.tokens * a.chunks;
  const int64_t most = (int64_t)ops_sm_count() * 2;
  const int grid = (int)(a.items < most ? a.items : most);
  auto* fn = a.rot == D ? (a.inter ? rotate_kernel<T, D, true, true> : rotate_kernel<T, D, false, true>)
                        : (a.inter ? rotate_kernel<T, D, true, false> : rotate_kernel<T, D, false, false>);
  return ops_launch(fn, grid, kWarps * 32, smem, 0, st, a);
}

template <typename T>
cudaError_t by_width(Args& a, int d, cudaStream_t st) {
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
  if (heads > (1 << 20)) return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: too many heads");
  if ((r->q_heads && (!r->q || !r->q_out)) || (r->rot && (!r->positions || !r->table)) ||
      (r->kv_heads && (!r->k || !r->v || !r->slots || (r->num_pages && (!r->k_pages || !r->v_pages)))))
    return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: NULL argument");
  if (r->kv_heads && (r->page_size < 1 || r->num_pages < 0))
    return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: page_size must be >= 1 and num_pages >= 0");
  if (r->rot && r->contexts < 0) return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: contexts must be >= 0");
  if (r->rot && !aligned(r->table, 16)) return api_fail(WFST_ERR_INVALID_ARG, "norm_rotate: arrays must be 16-byte aligned");
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
  a.capacity = r->kv_heads ? (int64_t)r->num_pages * r->page_size : 0;
  a.tokens = r->tokens, a.hq = r->q_heads, a.hkv = r->kv_heads, a.rot = r->rot;
  a.page = r->page_size, a.contexts = r->contexts, a.inter = r->interleaved != 0;
  a.eps = r->eps;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = r->dtype == WFST_F16 ? by_width<__half>(a, r->head_dim, st)
                                             : by_width<__nv_bfloat16>(a, r->head_dim, st);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "norm_rotate launch");
}
