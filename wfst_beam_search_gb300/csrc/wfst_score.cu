// wfst_score.cu — how likely given tokens are: log probabilities, entropy, the
// likeliest alternatives.
//
//   y_i = x_i - max x,  Z = sum exp y_i,  U = sum exp(y_i) y_i
//   logprob = y_t - log Z,  entropy = log Z - U / Z
//   alternatives: the k first by descending x, equal ones by ascending index
//
// A pass has to read the logits once; HBM bounds it with many rows.  A CTA takes a
// row, or with few rows a cluster of CTAs does, a part each.  A thread reads 16 bytes
// at a time, four of them ahead, and keeps the running maximum with Z and U against it;
// rows end with the CTA's (and the cluster's) threads putting theirs together.
//
// The alternatives cost no second pass.  A thread has its own largest logit: the k
// largest of those are k logits, so the k largest of all are among those not below the
// k-th of them, which only the threads that have one so large can hold.  What bound lets
// between k and some more threads through is found by halving; what they hold above it,
// read again (from the L2 cache), is usually a few more than k, and is ordered by
// counting.  Where it does not fit the list (many equal logits), the list is cut to its
// k first whenever it is full, and from then on only what is before the last of those
// goes in.
#include <cooperative_groups.h>

#include "wfst_ops.h"

namespace cg = cooperative_groups;

namespace wfst {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kList = 64 + kThreads * 8;  // candidates: what is kept, and what all threads' 16 bytes can add
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Args {
  const void* logits;
  const int32_t* tokens;
  float *logprobs, *entropy;
  int32_t* top_tokens;
  float* top_logprobs;
  int64_t stride;
  int32_t rows, vocab, top;
};

// Larger logit, larger key; -0 and +0 have one; 0: no logit (-inf, NaN).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return v > -INFINITY ? b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u) : 0u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }
// Order of the tokens: larger logit first, then lower index.
__device__ __forceinline__ uint64_t order_of(uint32_t key, int e) { return (uint64_t)key << 32 | (0xffffffffu - (uint32_t)e); }

__device__ __forceinline__ float exp2a(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// the larger one, NaN if either is
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Z and U (in powers of two) against the largest logit m.
struct Sums {
  float m = -INFINITY, z = 0.f, u = 0.f;
  // moves the reference up; what lies at -inf stays nothing
  __device__ __forceinline__ void raise(float to) {
    if (!(to > m)) return;
    if (m > -INFINITY) {
      const float down = (m - to) * kLog2e, f = exp2a(down);
      u = f > 0.f ? f * (u + down * z) : 0.f * u;  // (NaN stays)
      z *= f;
    }
    m = to;
  }
  __device__ __forceinline__ void add(const Sums& o) {
    Sums b = o;
    raise(b.m);
    b.raise(m);
    z += b.z;
    u += b.u;
  }
};

template <typename T>
struct Row {
  static constexpr int VEC = 16 / (int)sizeof(T);
  const T* p;
  int vocab, pad;  // pad: elements between the 16-byte boundary before p and p
  __device__ __forceinline__ bool inside(int i) const { return i * VEC - pad >= 0 && (i + 1) * VEC - pad <= vocab; }
  // granule i: elements [i * VEC - pad, i * VEC - pad + VEC), -inf outside
  __device__ __forceinline__ uint4 load(int i) const {
    const int e = i * VEC - pad;
    if (inside(i)) return *reinterpret_cast<const uint4*>(p + e);
    alignas(16) T v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; j++) v[j] = e + j >= 0 && e + j < vocab ? p[e + j] : from_f32<T>(-INFINITY);
    return *reinterpret_cast<const uint4*>(v);
  }
};
template <typename T>
__device__ __forceinline__ void widen(uint4 raw, float (&v)[16 / sizeof(T)]);
template <>
__device__ __forceinline__ void widen<float>(uint4 raw, float (&v)[4]) {
  v[0] = __uint_as_float(raw.x), v[1] = __uint_as_float(raw.y), v[2] = __uint_as_float(raw.z), v[3] = __uint_as_float(raw.w);
}
template <typename T>
__device__ __forceinline__ void widen(uint4 raw, float (&v)[16 / sizeof(T)]) {
  const float2 a = unpack2<T>(raw.x), b = unpack2<T>(raw.y), c = unpack2<T>(raw.z), d = unpack2<T>(raw.w);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
}

struct Shared {
  Sums part[kWarps];
  uint32_t least[kWarps], most[kWarps];
  Sums box[kMaxCluster];                       // the cluster's CTAs' sums
  uint64_t first[kMaxCluster * WFST_SCORE_TOP];  // and their first ones
  uint64_t list[kList], kept[WFST_SCORE_TOP];
  uint32_t best[kThreads];                     // each thread's largest logit
  uint16_t winner[kThreads];                   // threads that hold candidates
  uint32_t count, winners;
};

// The `top` first of list[0 .. n) in order, to `to` (0 where there are no more).
__device__ void order_list(const uint64_t* list, uint32_t n, uint64_t* to, int top) {
  for (int i = threadIdx.x; i < top; i += kThreads) to[i] = 0;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t v = list[i];
    int before = 0;
    for (uint32_t j = 0; j < n && before < top; j++) before += list[j] > v;
    if (before < top) to[before] = v;
  }
  __syncthreads();
}

// The `top` first logits among the granules [lo, hi) that this CTA has read, in order, to sh->kept.
template <typename T>
__device__ void alternatives(const Row<T>& row, int lo, int hi, int top, Shared* sh) {
  constexpr int VEC = Row<T>::VEC;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t mine = sh->best[tid];
  // ---- a bound that at least `top` threads' largest logits reach, and not many more if it can be
  uint32_t least = mine ? mine : ~0u, most = mine;
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) sh->least[warp] = least, sh->most[warp] = most;
  if (tid == 0) sh->count = sh->winners = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; w++) least = min(least, sh->least[w]), most = max(most, sh->most[w]);
  // at least `top` reach low, fewer reach high
  uint32_t low = least, high = most + 1;
  const int enough = top + top / 2 + 4;
  int n = __syncthreads_count(mine != 0);
  if (n < top) low = 1, n = 0;  // fewer threads have a logit: all logits are candidates
  while (n > enough && high - low > 1) {
    const uint32_t mid = low + (high - low) / 2;
    const int c = __syncthreads_count(mine >= mid);
    if (c >= top)
      low = mid, n = c;
    else
      high = mid;
  }
  // ---- the threads that reach it, in order
  const bool wins = mine != 0 && mine >= low;
  const uint32_t votes = __ballot_sync(0xffffffffu, wins);
  if (lane == 0) sh->least[warp] = __popc(votes);
  __syncthreads();
  uint32_t before = 0, winners = 0;
#pragma unroll
  for (int w = 0; w < kWarps; w++) before += w < warp ? sh->least[w] : 0, winners += sh->least[w];
  if (wins) sh->winner[before + __popc(votes & ((1u << lane) - 1))] = (uint16_t)tid;
  __syncthreads();
  // ---- what they have read, from the first granule on, again
  const int each = (hi - lo + kThreads - 1) / kThreads;
  const int items = each * (int)winners;
  auto visit = [&](int i, uint64_t after, auto push) {
    const int g = lo + i / (int)winners * kThreads + sh->winner[i % (int)winners];
    if (g >= hi) return;
    float v[VEC];
    widen<T>(row.load(g), v);
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      const uint32_t key = key_of(v[j]);
      if (key && key >= low) {
        const uint64_t o = order_of(key, g * VEC - row.pad + j);
        if (o > after) push(o);
      }
    }
  };
  for (int i = tid; i < items; i += kThreads)
    visit(i, 0, [&](uint64_t o) {
      const uint32_t at = atomicAdd(&sh->count, 1u);
      if (at < (uint32_t)kList) sh->list[at] = o;
    });
  __syncthreads();
  uint32_t found = sh->count;
  if (found > (uint32_t)kList / 2) {  // equal logits, mostly: in steps, the list cut to the first ones in between
    uint64_t after = 0;
    uint32_t have = 0;
    __syncthreads();
    for (int i0 = 0; i0 < items; i0 += kThreads) {
      if (tid == 0) sh->count = have;
      __syncthreads();
      if (i0 + tid < items) visit(i0 + tid, after, [&](uint64_t o) { sh->list[atomicAdd(&sh->count, 1u)] = o; });
      __syncthreads();
      found = have = sh->count;
      __syncthreads();
      if (found > (uint32_t)WFST_SCORE_TOP || i0 + kThreads >= items) {
        order_list(sh->list, found, sh->kept, top);
        if (tid < top) sh->list[tid] = sh->kept[tid];
        have = min(found, (uint32_t)top);
        if (have == (uint32_t)top) after = sh->kept[top - 1];
        __syncthreads();
      }
    }
    return;
  }
  order_list(sh->list, found, sh->kept, top);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) score_kernel(const Args a) {
  constexpr int VEC = Row<T>::VEC, kAhead = 4;
  extern __shared__ __align__(16) unsigned char raw[];
  Shared* sh = reinterpret_cast<Shared*>(raw);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank(), r = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  ops_begin();
  ops_next();
  Row<T> row;
  row.p = reinterpret_cast<const T*>(a.logits) + r * a.stride;
  row.vocab = a.vocab;
  row.pad = (int)(((uintptr_t)row.p & 15) / sizeof(T));
  const int granules = (a.vocab + row.pad + VEC - 1) / VEC, each = (granules + C - 1) / C;
  const int lo = min(rank * each, granules), hi = min(lo + each, granules);
  const int t = tid == 0 && rank == 0 ? ops_load(a.tokens + r) : 0;
  const float x_t = tid == 0 && rank == 0 && t >= 0 && t < a.vocab ? to_f32(ops_load(row.p + t)) : 0.f;

  // ---- one pass
  Sums s;
  for (int i0 = lo + tid; i0 < hi; i0 += kAhead * kThreads) {
    uint4 raw[kAhead];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      const int i = i0 + j * kThreads;
      raw[j] = make_uint4(0, 0, 0, 0);
      if (i < hi) raw[j] = row.load(i);
    }
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      if (i0 + j * kThreads >= hi) break;
      float v[VEC];
      widen<T>(raw[j], v);
#pragma unroll
      for (int e = 0; e < VEC; e++) top = fmaxf(top, v[e]);
    }
    s.raise(top);
    const float ref = s.m > -INFINITY ? s.m : 0.f;
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      if (i0 + j * kThreads >= hi) break;
      float v[VEC];
      widen<T>(raw[j], v);
#pragma unroll
      for (int e = 0; e < VEC; e++) {
        // (from 2^-1000 on it weighs nothing, and must not be -inf: 0 times that is NaN)
        const float y = max_or_nan((v[e] - ref) * kLog2e, -1000.f), w = exp2a(y);
        s.z += w;
        s.u += w * y;
      }
    }
  }
  sh->best[tid] = key_of(s.m);
#pragma unroll
  for (int x = 16; x; x /= 2) {
    Sums o;
    o.m = __shfl_xor_sync(0xffffffffu, s.m, x);
    o.z = __shfl_xor_sync(0xffffffffu, s.z, x);
    o.u = __shfl_xor_sync(0xffffffffu, s.u, x);
    s.add(o);
  }
  if (lane == 0) sh->part[warp] = s;
  __syncthreads();
  if (a.top) alternatives(row, lo, hi, a.top, sh);
  const uint64_t* first = sh->kept;
  Sums all = sh->part[0];
#pragma unroll
  for (int w = 1; w < kWarps; w++) all.add(sh->part[w]);
  if (C > 1) {
    cl.sync();  // every CTA runs
    Shared* to = cl.map_shared_rank(sh, 0);
    if (tid == 0) to->box[rank] = all;
    if (tid < a.top) to->first[rank * a.top + tid] = sh->kept[tid];
    cl.sync();
    if (rank) return;
    all = sh->box[0];
    for (int w = 1; w < C; w++) all.add(sh->box[w]);
    if (a.top) order_list(sh->first, C * a.top, sh->kept, a.top);
  }
  // (NaN and +inf: Z is NaN; no logit: Z is 0)
  const float log_z = logf(all.z), ref = all.m > -INFINITY ? all.m : 0.f;
  if (tid == 0) {
    float v = 0.f;
    if (t >= a.vocab)
      v = NAN;
    else if (t >= 0)
      v = all.z == 0.f ? -INFINITY : x_t - ref - log_z;
    a.logprobs[r] = v;
    a.entropy[r] = all.z == 0.f ? 0.f : log_z - all.u / all.z * kLn2;
  }
  for (int i = tid; i < a.top; i += kThreads) {
    const uint64_t o = first[i];
    a.top_tokens[(int64_t)r * a.top + i] = o ? (int)(0xffffffffu - (uint32_t)o) : -1;
    a.top_logprobs[(int64_t)r * a.top + i] = o ? of_key((uint32_t)(o >> 32)) - ref - log_z : -INFINITY;
  }
}

template <typename T>
cudaError_t launch(const Args& a, cudaStream_t st) {
  // A row is shared among as many CTAs as leave each of them a few rounds and all of them a
  // place: some four to a multiprocessor are resident.
  const int granules = (int)(((int64_t)a.vocab * sizeof(T) + 15) / 16);
  int C = 1;
  while (C < kMaxCluster && granules / C > 2 * kThreads && (int64_t)a.rows * C * 2 <= 4 * ops_sm_count()) C *= 2;
  return ops_launch(score_kernel<T>, dim3((unsigned)a.rows * C), kThreads, (int)sizeof(Shared), C, st, a);
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
  if (r->rows > INT32_MAX / kMaxCluster) return api_fail(WFST_ERR_INVALID_ARG, "score_tokens: too many rows");
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
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = r->dtype == WFST_F32   ? launch<float>(a, st)
                        : r->dtype == WFST_F16 ? launch<__half>(a, st)
                                               : launch<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "score_tokens launch");
}
