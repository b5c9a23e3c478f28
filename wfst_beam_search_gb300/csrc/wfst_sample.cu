// wfst_sample.cu — the next token of each lane, drawn from its logits with one
// given uniform number.
//
//   y_i = (x_i - max x) / T,  w_i = exp(y_i)
//   order: descending x, equal ones by ascending index; kept is the shortest of
//   three prefixes of it: the first k; the shortest whose weight reaches
//   p * (weight of the first k); those with w_i >= min_p
//   token: the first index, in index order, whose cumulative kept weight
//   exceeds u * total;  logprob = y_token - log(total)
//   (-inf and NaN logits weigh nothing; a lane with no other logit gets token
//   -1, logprob -inf and kept 0; T = 0 takes the first largest logit)
//
// Weights are summed as whole multiples of 2^-43 of the largest one, in 64
// bits: a sum then has one value in any order, so a token depends neither on
// how the row is split nor on the order of atomics, and a row of 2^20 logits
// still fits.  Weights themselves are fp32 (the plain expf).
//
// A pass has to read the logits once, which takes microseconds; what bounds it
// is the chain of row-wide decisions (largest logit, k-th logit, total weight,
// weight's threshold, drawn token).  A cluster of CTAs takes one row, so a
// decision costs a cluster barrier and not a launch.  Thresholds come from
// radix selection on the logits' ordered bits, 11 bits a level, over counts
// (k) or weights (p): no sort.
#include <cooperative_groups.h>

#include "wfst_ops.h"

namespace cg = cooperative_groups;

namespace wfst {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kFixed = 43;

struct Args {
  const void* logits;
  const float *u, *temp_v, *top_p_v, *min_p_v;
  const int32_t* top_k_v;
  int32_t* token;
  float* logprob;
  int32_t* kept;
  int64_t stride;
  int32_t vocab, top_k;
  float temp, top_p, min_p;
};

// NaN counts as -inf; -0 and +0 are equal.
__device__ __forceinline__ float canonical(float v) { return v == v ? v + 0.f : -INFINITY; }
// Larger logit, larger key.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
// floor(w * 2^43) of 0 <= w <= 1
__device__ __forceinline__ uint64_t fixed_of(float w) {
  const uint32_t b = __float_as_uint(w);
  const uint32_t sh = 127u - (b >> 23);
  const uint64_t m = (uint64_t)((b & 0x7fffffu) | 0x800000u) << (kFixed - 23);
  return sh < 64u ? m >> sh : 0;
}

template <typename T>
struct Row {
  static constexpr int VEC = 16 / (int)sizeof(T);
  const T* p;
  int vocab, pad;  // pad: elements between the 16-byte boundary before p and p
  // granule i: elements [i * VEC - pad, i * VEC - pad + VEC), -inf outside
  __device__ __forceinline__ void load(int i, float (&v)[VEC]) const {
    const int e = i * VEC - pad;
    if (e >= 0 && e + VEC <= vocab) {
      const uint4 raw = *reinterpret_cast<const uint4*>(p + e);
      const T* r = reinterpret_cast<const T*>(&raw);
#pragma unroll
      for (int j = 0; j < VEC; j++) v[j] = canonical(to_f32(r[j]));
    } else {
#pragma unroll
      for (int j = 0; j < VEC; j++) v[j] = e + j >= 0 && e + j < vocab ? canonical(to_f32(p[e + j])) : -INFINITY;
    }
  }
  __device__ __forceinline__ bool has(int i, int j) const {
    const int e = i * VEC - pad + j;
    return e >= 0 && e < vocab;
  }
};

struct Shared {
  uint32_t count[2][kBins];
  unsigned long long weight[2][kBins];
  unsigned long long warp_a[4][kWarps];  // one row per use: a reader is never overtaken
  uint32_t warp_b[4][kWarps];
  float top[kWarps];
  uint32_t scan_c[kWarps];
  unsigned long long scan_w[kWarps];
  uint32_t bin;
  unsigned long long above;
};

// From the largest bin down, the first one where the running sum reaches
// `want` (1 <= want <= the bins' sum); *above is the sum before it.  Every CTA
// of the cluster adds up all CTAs' bins and finds the same.
template <typename V>
__device__ __forceinline__ uint32_t find_bin(cg::cluster_group& cl, V* bins, unsigned long long want, Shared* sh,
                                             unsigned long long* above) {
  constexpr int P = kBins / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned long long v[P], mine = 0;
#pragma unroll
  for (int i = 0; i < P; i++) v[i] = 0;
  const int top = kBins - 1 - tid * P;  // this thread's bins: top, top - 1, ...
  for (unsigned r = 0; r < cl.num_blocks(); r++) {
    const V* b = cl.map_shared_rank(bins, r);
#pragma unroll
    for (int i = 0; i < P; i++) v[i] += b[top - i];
  }
#pragma unroll
  for (int i = 0; i < P; i++) mine += v[i];
  unsigned long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const unsigned long long up = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += up;
  }
  if (lane == 31) sh->scan_w[warp] = incl;
  __syncthreads();
  unsigned long long before = incl - mine;
  for (int w = 0; w < warp; w++) before += sh->scan_w[w];
  if (before < want && want <= before + mine) {
    unsigned long long run = before;
#pragma unroll
    for (int i = 0; i < P; i++) {
      if (run < want && want <= run + v[i]) {
        sh->bin = top - i;
        sh->above = run;
      }
      run += v[i];
    }
  }
  __syncthreads();
  const uint32_t bin = sh->bin;
  *above = sh->above;
  __syncthreads();
  return bin;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char raw_smem[];
  Shared* sh = reinterpret_cast<Shared*>(raw_smem);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int VEC = Row<T>::VEC;
  Row<T> row;
  row.p = reinterpret_cast<const T*>(a.logits) + b * a.stride;
  row.vocab = a.vocab;
  row.pad = (int)(((uintptr_t)row.p & 15) / sizeof(T));
  const int granules = (a.vocab + row.pad + VEC - 1) / VEC;
  // each warp of the cluster has a run of granules, in index order
  const int parts = C * kWarps, part = rank * kWarps + warp;
  const int lo = (int)((int64_t)granules * part / parts), hi = (int)((int64_t)granules * (part + 1) / parts);

  float temp = a.temp_v ? a.temp_v[b] : a.temp;
  int k = a.top_k_v ? a.top_k_v[b] : a.top_k;
  const float top_p = a.top_p_v ? a.top_p_v[b] : a.top_p;
  const float min_p = fminf(a.min_p_v ? a.min_p_v[b] : a.min_p, 1.f);
  if (!(temp > 0.f)) {
    temp = 1.f;
    k = 1;
  }
  const float inv_t = 1.f / temp;
  const bool by_k = k > 0 && k < a.vocab, by_p = top_p < 1.f || top_p != top_p;

  // ---- the largest logit
  float top = -INFINITY;
  for (int i = lo + lane; i < hi; i += 32) {
    float v[VEC];
    row.load(i, v);
#pragma unroll
    for (int j = 0; j < VEC; j++) top = fmaxf(top, v[j]);
  }
#pragma unroll
  for (int x = 16; x; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  if (lane == 0) sh->top[warp] = top;
  for (int i = tid; i < kBins; i += kThreads) {
    sh->count[0][i] = sh->count[1][i] = 0;
    sh->weight[0][i] = sh->weight[1][i] = 0;
  }
  cl.sync();
  for (int i = lane; i < parts; i += 32) top = fmaxf(top, *cl.map_shared_rank(&sh->top[i % kWarps], i / kWarps));
#pragma unroll
  for (int x = 16; x; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  if (top == -INFINITY) {  // nothing to draw from (the same for the whole cluster)
    if (rank == 0 && tid == 0) {
      a.token[b] = -1;
      a.logprob[b] = -INFINITY;
      a.kept[b] = 0;
    }
    cl.sync();
    return;
  }
  auto y_of = [&](float x) { return x == top ? 0.f : (x - top) * inv_t; };
  auto w_of = [&](float x) { return fixed_of(expf(y_of(x))); };

  // kept so far: key > cut, or key == cut and among its first `ties` by index
  uint32_t cut = 0;
  uint64_t ties = UINT64_MAX;

  auto clear_bins = [&](int buf) {
    for (int i = tid; i < kBins; i += kThreads) {
      sh->count[buf][i] = 0;
      sh->weight[buf][i] = 0;
    }
  };

  int buf = 0;
  // ---- the k-th logit
  if (by_k) {
    uint32_t prefix = 0, mask = 0;
    uint64_t want = (uint64_t)k;
    for (int level = 0; level < 3; level++) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
      const uint32_t width = level == 2 ? 0x3ffu : 0x7ffu;
      for (int i = lo + lane; i < hi; i += 32) {
        float v[VEC];
        row.load(i, v);
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          const uint32_t key = key_of(v[j]);
          if (row.has(i, j) && (key & mask) == prefix) atomicAdd(&sh->count[buf][key >> shift & width], 1u);
        }
      }
      cl.sync();
      unsigned long long above;
      const uint32_t bin = find_bin(cl, sh->count[buf], want, sh, &above);
      want -= above;
      prefix |= bin << shift;
      mask |= width << shift;
      buf ^= 1;  // the other buffer is clean, and cleared again once no one reads it
      if (level < 2) {
        // the buffer of the level before last: everyone has passed this level's barrier since
        if (level == 1) clear_bins(buf);
        __syncthreads();
      }
    }
    cut = prefix;
    ties = want;
    cl.sync();
    clear_bins(0);
    clear_bins(1);
    __syncthreads();
  }

  // ---- the weight that is kept
  if (by_p) {
    uint64_t sum = 0;
    for (int i = lo + lane; i < hi; i += 32) {
      float v[VEC];
      row.load(i, v);
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const uint32_t key = key_of(v[j]);
        if (!by_k || key > cut) sum += w_of(v[j]);
      }
    }
#pragma unroll
    for (int x = 16; x; x /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (lane == 0) sh->warp_a[0][warp] = sum;
    cl.sync();
    sum = 0;
    for (int i = lane; i < parts; i += 32) sum += *cl.map_shared_rank(&sh->warp_a[0][i % kWarps], i / kWarps);
#pragma unroll
    for (int x = 16; x; x /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (by_k) sum += ties * w_of(of_key(cut));
    const double goal = ceil((double)sum * (double)top_p);
    uint64_t want = goal >= 1.0 ? (uint64_t)goal : 1;
    if (want > sum) want = sum;
    uint32_t prefix = 0, mask = 0;
    buf = 0;
    for (int level = 0; level < 3; level++) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
      const uint32_t width = level == 2 ? 0x3ffu : 0x7ffu;
      for (int i = lo + lane; i < hi; i += 32) {
        float v[VEC];
        row.load(i, v);
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          const uint32_t key = key_of(v[j]);
          if ((key & mask) == prefix && key >= cut) {
            const uint64_t w = w_of(v[j]);
            if (w) atomicAdd(&sh->weight[buf][key >> shift & width], (unsigned long long)w);
          }
        }
      }
      cl.sync();
      unsigned long long above;
      const uint32_t bin = find_bin(cl, sh->weight[buf], want, sh, &above);
      want -= above;
      prefix |= bin << shift;
      mask |= width << shift;
      buf ^= 1;
      if (level < 2) {
        if (level == 1) clear_bins(buf);
        __syncthreads();
      }
    }
    const uint64_t each = w_of(of_key(prefix));
    const uint64_t need = (want + each - 1) / each;
    if (!by_k || prefix > cut) {
      cut = prefix;
      ties = need;
    } else {
      ties = need < ties ? need : ties;
    }
  }

  // ---- where the equal logits end that are kept
  int last = INT32_MAX;
  if (by_k || by_p) {
    uint32_t n = 0;
    for (int i = lo + lane; i < hi; i += 32) {
      float v[VEC];
      row.load(i, v);
#pragma unroll
      for (int j = 0; j < VEC; j++) n += row.has(i, j) && key_of(v[j]) == cut;
    }
#pragma unroll
    for (int x = 16; x; x /= 2) n += __shfl_xor_sync(0xffffffffu, n, x);
    if (lane == 0) sh->warp_b[0][warp] = n;
    cl.sync();
    uint64_t before = 0;
    int at = -1;
    uint64_t left = 0;
    for (int i = 0; i < parts; i++) {  // every thread the same
      const uint32_t c = *cl.map_shared_rank(&sh->warp_b[0][i % kWarps], i / kWarps);
      if (at < 0 && before + c >= ties) {
        at = i;
        left = ties - before;
      }
      before += c;
    }
    if (before > ties) {
      // walk the run of granules that holds the last kept one
      const int w_lo = (int)((int64_t)granules * at / parts), w_hi = (int)((int64_t)granules * (at + 1) / parts);
      for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
        const int i = i0 + lane;
        float v[VEC];
        uint32_t mine = 0;
        if (i < w_hi) {
          row.load(i, v);
#pragma unroll
          for (int j = 0; j < VEC; j++) mine += row.has(i, j) && key_of(v[j]) == cut;
        }
        uint32_t incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const uint32_t up = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += up;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
        if (left > all) {
          left -= all;
          continue;
        }
        int found = INT32_MAX;
        if (mine && incl >= left && incl - mine < left) {
          uint32_t c = incl - mine;
#pragma unroll
          for (int j = 0; j < VEC; j++)
            if (row.has(i, j) && key_of(v[j]) == cut && ++c == left) found = i * VEC - row.pad + j;
        }
#pragma unroll
        for (int x = 16; x; x /= 2) found = min(found, __shfl_xor_sync(0xffffffffu, found, x));
        last = found;
        break;
      }
    }
  }

  // ---- the draw
  auto keeps = [&](int i, int j, float x, uint64_t* w) {
    *w = 0;
    if (!row.has(i, j)) return false;
    const uint32_t key = key_of(x);
    if (key < cut || (key == cut && i * VEC - row.pad + j > last)) return false;
    const float e = expf(y_of(x));
    if (e < min_p) return false;
    *w = fixed_of(e);
    return true;
  };
  uint64_t sum = 0;
  uint32_t n = 0;
  for (int i = lo + lane; i < hi; i += 32) {
    float v[VEC];
    row.load(i, v);
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      uint64_t w;
      n += keeps(i, j, v[j], &w);
      sum += w;
    }
  }
#pragma unroll
  for (int x = 16; x; x /= 2) {
    sum += __shfl_xor_sync(0xffffffffu, sum, x);
    n += __shfl_xor_sync(0xffffffffu, n, x);
  }
  if (lane == 0) {
    sh->warp_a[1][warp] = sum;
    sh->warp_b[1][warp] = n;
  }
  cl.sync();
  uint64_t total = 0;
  uint32_t kept = 0;
  for (int i = 0; i < parts; i++) {
    total += *cl.map_shared_rank(&sh->warp_a[1][i % kWarps], i / kWarps);
    kept += *cl.map_shared_rank(&sh->warp_b[1][i % kWarps], i / kWarps);
  }
  const float u = a.u[b];
  const double goal = (double)u * (double)total;
  uint64_t aim = goal > 0.0 ? (goal < 9.0e18 ? (uint64_t)goal : UINT64_MAX) : 0;
  if (aim > total - 1) aim = total - 1;
  uint64_t before = 0;
  int at = 0;
  for (int i = 0; i < parts; i++) {
    const uint64_t w = *cl.map_shared_rank(&sh->warp_a[1][i % kWarps], i / kWarps);
    if (before + w > aim) {
      at = i;
      break;
    }
    before += w;
  }
  if (at == part) {
    uint64_t left = aim - before;  // the first element whose running sum exceeds it
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      float v[VEC];
      uint64_t w[VEC], mine = 0;
      if (i < hi) {
        row.load(i, v);
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          keeps(i, j, v[j], &w[j]);
          mine += w[j];
        }
      }
      uint64_t incl = mine;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const uint64_t up = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += up;
      }
      const uint64_t all = __shfl_sync(0xffffffffu, incl, 31);
      if (all <= left) {
        left -= all;
        continue;
      }
      if (incl > left && incl - mine <= left) {
        uint64_t run = incl - mine;
        bool done = false;
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          run += w[j];
          if (!done && run > left) {
            done = true;
            a.token[b] = i * VEC - row.pad + j;
            a.logprob[b] = y_of(v[j]) - (float)log((double)total * (1.0 / (1ull << kFixed)));
            a.kept[b] = (int32_t)kept;
          }
        }
      }
      break;
    }
  }
  cl.sync();  // no CTA leaves while another may read its shared memory
}

template <typename T>
cudaError_t launch(const Args& a, int lanes, cudaStream_t st) {
  int c = 1;
  while (c < kMaxCluster && a.vocab > 8192 * c) c *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)lanes * c);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
  return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, sample_kernel<T>, a) : e;
}

}  // namespace
}  // namespace wfst

using namespace wfst;

extern "C" int wfst_sample_tokens(const wfst_sample_args* r, void* stream) {
  if (!r) return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: NULL argument");
  if (r->dtype != WFST_F32 && r->dtype != WFST_F16 && r->dtype != WFST_BF16)
    return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: bad dtype");
  if (r->lanes < 0 || r->lanes > (1 << 27)) return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: lanes out of range");
  if (r->vocab < 1 || r->vocab > (1 << 20)) return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: vocab must be in [1, 2^20]");
  if (r->lanes > 1 && r->stride < r->vocab) return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: stride must be >= vocab");
  if (!r->temperature_v && !(r->temperature >= 0.f && r->temperature <= 3.0e38f))
    return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: temperature must be >= 0");
  if (!r->top_k_v && r->top_k < 0) return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: top_k must be >= 0");
  if (!r->top_p_v && !(r->top_p > 0.f)) return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: top_p must be > 0");
  if (!r->min_p_v && !(r->min_p >= 0.f && r->min_p <= 1.f))
    return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: min_p must be in [0, 1]");
  if (r->lanes == 0) return WFST_OK;
  if (!r->logits || !r->uniform || !r->tokens || !r->logprobs || !r->kept)
    return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: NULL argument");
  const size_t size = r->dtype == WFST_F32 ? 4 : 2;
  if (!aligned(r->logits, size)) return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: logits not aligned to their type");
  const int dev = ops_device({r->logits, r->uniform, r->temperature_v, r->top_k_v, r->top_p_v, r->min_p_v, r->tokens,
                              r->logprobs, r->kept});
  if (dev < 0) return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: every array must be device memory of one device");
  OpsDevice guard(dev);
  Args a;
  a.logits = r->logits, a.u = r->uniform;
  a.temp_v = r->temperature_v, a.top_k_v = r->top_k_v, a.top_p_v = r->top_p_v, a.min_p_v = r->min_p_v;
  a.token = r->tokens, a.logprob = r->logprobs, a.kept = r->kept;
  a.stride = r->stride, a.vocab = r->vocab;
  a.temp = r->temperature, a.top_k = r->top_k, a.top_p = r->top_p, a.min_p = r->min_p;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = r->dtype == WFST_F32   ? launch<float>(a, r->lanes, st)
                        : r->dtype == WFST_F16 ? launch<__half>(a, r->lanes, st)
                                               : launch<__nv_bfloat16>(a, r->lanes, st);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "sample_tokens launch");
}
