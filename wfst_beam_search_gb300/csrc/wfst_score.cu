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
// The alternatives cost no second pass.  A thread keeps the largest logit of each
// eighth of what it reads.  The k largest of the threads' largest logits are k logits,
// so the k largest of all are among those not below the k-th of them.  A bound that k
// threads reach, and not many more, is found by halving; the eighths that reach it, read
// again, hold a few more than k logits above it, usually, which are ordered by counting.
// Where they do not fit the list (many equal logits), the list is cut to its k first
// whenever it is full, and from then on only what is before the last of those goes in.
//
// 16-bit logits are compared two by two, and fp32 arithmetic is on two at a time: with one
// at a time the instructions bound it (2048 x 131072, bf16, 110 us without alternatives,
// two at a time and eight granules ahead 83).  2048 x 131072, bf16, with 20 alternatives
// takes 94 us (5.7 TB/s), 2000 x 20000, fp16, 21, 64 x 131071 with 8 10.1, 1 x 5000, fp32,
// with 5 5.5; the short ones are bound by the chain of steps after the pass.
#include <cooperative_groups.h>

#include <type_traits>

#include "wfst_ops.h"

namespace cg = cooperative_groups;

namespace wfst {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kAhead = 8;   // granules of 16 bytes that a thread loads at once (four: 2048 x 131072 95 us, eight 83)
constexpr int kParts = 8;   // of what a thread reads, each with its largest logit
constexpr float kLog2e = 1.4426950408889634f;

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

// Z and U against the largest logit m.
struct Sums {
  float m = -INFINITY, z = 0.f, u = 0.f;
  // moves the reference up; what lies at -inf stays nothing
  __device__ __forceinline__ void raise(float to) {
    if (!(to > m)) return;
    if (m > -INFINITY) {
      const float down = fmaxf(m - to, -1000.f), f = exp2a(down * kLog2e);
      u = f * (u + down * z);
      z *= f;
    }
    m = to;
  }
  // all lanes get the sum over the warp
  __device__ __forceinline__ void over_warp() {
    const uint32_t top = __reduce_max_sync(0xffffffffu, key_of(m));
    if (top) raise(of_key(top));
#pragma unroll
    for (int x = 16; x; x /= 2) z += __shfl_xor_sync(0xffffffffu, z, x), u += __shfl_xor_sync(0xffffffffu, u, x);
    m = top ? of_key(top) : -INFINITY;
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

template <int N>  // threads
struct Shared {
  static constexpr int kList = WFST_SCORE_TOP + N * 8;  // candidates: what is kept, and what all threads' 16 bytes can add
  Sums sums[N / 32];
  Sums box[kMaxCluster];                         // the cluster's CTAs' sums
  uint64_t first[kMaxCluster * WFST_SCORE_TOP];  // and their first ones
  uint64_t list[kList], kept[WFST_SCORE_TOP];
  uint32_t best[N], best_of[kParts][N];          // each thread's largest logit, and that of its parts
  uint16_t cell[kParts * N];                     // parts that hold candidates
  uint32_t cells, count, low;
};

// The `top` first of list[0 .. n) in order, to `to` (0 where there are no more).
template <int N>
__device__ void order_list(const uint64_t* list, uint32_t n, uint64_t* to, int top) {
  for (int i = threadIdx.x; i < top; i += N) to[i] = 0;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < n; i += N) {
    const uint64_t v = list[i];
    int before = 0;
#pragma unroll 8
    for (uint32_t j = 0; j < n; j++) before += list[j] > v;
    if (before < top) to[before] = v;
  }
  __syncthreads();
}

// The `top` first logits among the granules [lo, hi) that this CTA has read in parts of 2^steps
// granules a thread, in order, to sh->kept.
template <typename T, int N>
__device__ void alternatives(const Row<T>& row, int lo, int hi, int steps, int top, Shared<N>* sh) {
  constexpr int VEC = Row<T>::VEC, W = N / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // ---- a bound that at least `top` threads' largest logits reach, and not many more if it can be
  if (warp == 0) {
    uint32_t k[W], least = ~0u, most = 0, with = 0;
#pragma unroll
    for (int w = 0; w < W; w++) {
      k[w] = sh->best[w * 32 + lane];
      least = min(least, k[w] ? k[w] : ~0u), most = max(most, k[w]);
      with += k[w] != 0;
    }
    least = __reduce_min_sync(0xffffffffu, least), most = __reduce_max_sync(0xffffffffu, most);
    int n = (int)__reduce_add_sync(0xffffffffu, with);
    uint32_t low = least, high = most + 1;  // at least `top` reach low, fewer reach high
    if (n < top) low = 1, n = 0;            // fewer threads have a logit: all logits are candidates
    const int enough = top + top / 2 + 4;
    constexpr uint32_t kUnit = sizeof(T) == 4 ? 1u : std::is_same_v<T, __half> ? 1u << 13 : 1u << 16;  // between two values of T
    while (n > enough && high - low > kUnit) {
      const uint32_t mid = low + (high - low) / 2;
      uint32_t c = 0;
#pragma unroll
      for (int w = 0; w < W; w++) c += k[w] >= mid;
      c = __reduce_add_sync(0xffffffffu, c);
      if ((int)c >= top)
        low = mid, n = (int)c;
      else
        high = mid;
    }
    if (lane == 0) sh->low = low, sh->count = sh->cells = 0;
  }
  __syncthreads();
  const uint32_t low = sh->low;
  // ---- the parts that reach it
  if (sh->best[tid] >= low) {
    uint32_t reach = 0;
#pragma unroll
    for (int g = 0; g < kParts; g++) reach |= (sh->best_of[g][tid] >= low ? 1u : 0u) << g;
    for (uint32_t at = atomicAdd(&sh->cells, __popc(reach)); reach; reach &= reach - 1, at++)
      sh->cell[at] = (uint16_t)((__ffs(reach) - 1) * N + tid);
  }
  __syncthreads();
  // ---- what they hold: bits of a granule's logits that count, and one of them
  auto those = [&](const float (&v)[VEC], int g, uint64_t after) {
    uint32_t is = 0;
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      const uint32_t key = key_of(v[j]);
      is |= (key && key >= low && order_of(key, g * VEC - row.pad + j) > after ? 1u : 0u) << j;
    }
    return is;
  };
  constexpr uint32_t kList = Shared<N>::kList;
  auto push = [&](const float (&v)[VEC], int g, uint32_t is) {
    uint32_t at = is ? atomicAdd(&sh->count, __popc(is)) : 0;
#pragma unroll
    for (int j = 0; j < VEC; j++)
      if (is >> j & 1) {
        if (at < kList) sh->list[at] = order_of(key_of(v[j]), g * VEC - row.pad + j);
        at++;
      }
  };
  for (int i = tid; i < (int)sh->cells << steps; i += N) {
    const int c = sh->cell[i >> steps], g = lo + c % N + ((c / N << steps) + (i & ((1 << steps) - 1))) * N;
    if (g >= hi) continue;
    float v[VEC];
    widen<T>(row.load(g), v);
    push(v, g, those(v, g, 0));
  }
  __syncthreads();
  uint32_t found = sh->count;
  if (found <= kList / 2) {
    order_list<N>(sh->list, found, sh->kept, top);
    return;
  }
  // equal logits, mostly: everything again in order, the list cut to the first ones in between
  uint64_t after = 0;
  uint32_t have = 0;
  for (int i0 = lo; i0 < hi; i0 += N) {
    __syncthreads();
    if (tid == 0) sh->count = have;
    __syncthreads();
    if (i0 + tid < hi) {
      float v[VEC];
      widen<T>(row.load(i0 + tid), v);
      push(v, i0 + tid, those(v, i0 + tid, after));
    }
    __syncthreads();
    found = have = sh->count;
    if (found > (uint32_t)WFST_SCORE_TOP || i0 + N >= hi) {
      order_list<N>(sh->list, found, sh->kept, top);
      if (tid < top) sh->list[tid] = sh->kept[tid];
      have = min(found, (uint32_t)top);
      if (have == (uint32_t)top) after = sh->kept[top - 1];
    }
  }
  __syncthreads();
}

// ---- 16-bit logits two by two
template <typename T>
struct Pairs;
template <>
struct Pairs<__half> {
  using V = __half2;
  static constexpr uint32_t kNone = 0xfc00fc00u, kBound = 0xfbfffbffu;  // -inf; -65504
  static constexpr float kFrom = -32000.f;
};
template <>
struct Pairs<__nv_bfloat16> {
  using V = __nv_bfloat162;
  static constexpr uint32_t kNone = 0xff80ff80u, kBound = 0xf14af14au;  // -inf; -1e30
  static constexpr float kFrom = -1e29f;
};
template <typename V>
__device__ __forceinline__ V as(uint32_t w) {
  return *reinterpret_cast<const V*>(&w);
}
template <typename V>
__device__ __forceinline__ uint32_t bits(V v) {
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint64_t two(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 parts(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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

// The largest of some granules' logits; NaN is passed over.
template <typename T>
__device__ __forceinline__ float largest(const uint4 (&raw)[kAhead]) {
  if constexpr (sizeof(T) == 4) {
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kAhead; j++)
      top = fmaxf(fmaxf(fmaxf(top, __uint_as_float(raw[j].x)), fmaxf(__uint_as_float(raw[j].y), __uint_as_float(raw[j].z))),
                  __uint_as_float(raw[j].w));
    return top;
  } else {
    using V = typename Pairs<T>::V;
    V top = as<V>(Pairs<T>::kNone);
#pragma unroll
    for (int j = 0; j < kAhead; j++)
      top = __hmax2(__hmax2(top, __hmax2(as<V>(raw[j].x), as<V>(raw[j].y))), __hmax2(as<V>(raw[j].z), as<V>(raw[j].w)));
    const float2 t = unpack2<T>(bits(top));
    return fmaxf(t.x, t.y);
  }
}

// Adds some granules' logits, none of which is above s.m.
template <typename T>
__device__ __forceinline__ void add_granules(Sums& s, const uint4 (&raw)[kAhead]) {
  constexpr int VEC = Row<T>::VEC;
  // -inf weighs nothing, and must not be multiplied by that: it is brought up to a bound far below
  // the largest logit, where the weight is zero all the same
  if (constexpr float from = sizeof(T) == 4 ? -1e29f : Pairs<std::conditional_t<sizeof(T) == 4, __half, T>>::kFrom; s.m > from) {
    const uint64_t less = two(-s.m, -s.m), by = two(kLog2e, kLog2e);
    uint64_t z = two(0.f, 0.f), u = z;
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
      for (int e = 0; e < VEC / 2; e++) {
        float2 x;
        if constexpr (sizeof(T) == 4) {
          x = make_float2(max_or_nan(__uint_as_float(w[2 * e]), -1e30f), max_or_nan(__uint_as_float(w[2 * e + 1]), -1e30f));
        } else {
          using V = typename Pairs<T>::V;
          x = unpack2<T>(bits(__hmax2_nan(as<V>(w[e]), as<V>(Pairs<T>::kBound))));
        }
        const uint64_t y = add2(two(x.x, x.y), less);
        const float2 p = parts(mul2(y, by));
        const uint64_t f = two(exp2a(p.x), exp2a(p.y));
        z = add2(z, f);
        u = fma2(f, y, u);
      }
    }
    const float2 zz = parts(z), uu = parts(u);
    s.z += zz.x + zz.y;
    s.u += uu.x + uu.y;
  } else {  // a row of such logits alone, so far
    const float ref = s.m > -INFINITY ? s.m : 0.f;
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      float v[VEC];
      widen<T>(raw[j], v);
#pragma unroll
      for (int e = 0; e < VEC; e++) {
        const float y = max_or_nan(v[e] - ref, -1000.f), f = exp2a(y * kLog2e);
        s.z += f;
        s.u += f * y;
      }
    }
  }
}

// N threads: 128 for many short rows.
template <typename T, int N>
__global__ void __launch_bounds__(N, 1024 / N) score_kernel(const Args a) {
  constexpr int VEC = Row<T>::VEC, W = N / 32, A = kAhead;
  extern __shared__ __align__(16) unsigned char smem[];
  Shared<N>* sh = reinterpret_cast<Shared<N>*>(smem);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank(), r = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (C > 1) cl.barrier_arrive();  // (waited for where another CTA's memory is written)
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

  // ---- one pass, in parts of 2^rounds rounds of A granules
  int rounds = 0;
  while ((A * N * kParts) << rounds < hi - lo) rounds++;
  Sums s;
  uint32_t best = 0;
#pragma unroll 1
  for (int g = 0; g < kParts; g++) {
    float top_of = -INFINITY;
    for (int k = 0; k < 1 << rounds; k++) {
      const int i0 = lo + tid + ((g << rounds) + k) * (A * N);
      if (i0 >= hi) break;
      uint4 raw[A];
#pragma unroll
      for (int j = 0; j < kAhead; j++) {
        constexpr uint32_t kNone = sizeof(T) == 4 ? 0xff800000u : Pairs<std::conditional_t<sizeof(T) == 4, __half, T>>::kNone;
        raw[j] = make_uint4(kNone, kNone, kNone, kNone);
        if (i0 + j * N < hi) raw[j] = row.load(i0 + j * N);
      }
      const float top = largest<T>(raw);
      top_of = fmaxf(top_of, top);
      s.raise(top);
      add_granules<T>(s, raw);
    }
    const uint32_t key = key_of(top_of);
    sh->best_of[g][tid] = key;
    best = max(best, key);
  }
  sh->best[tid] = best;
  s.over_warp();
  if (lane == 0) sh->sums[warp] = s;
  __syncthreads();
  if (a.top) alternatives<T, N>(row, lo, hi, rounds + 3, a.top, sh);
  s = lane < W ? sh->sums[lane] : Sums();
  s.over_warp();
  if (C > 1) {
    cl.barrier_wait();  // every CTA runs
    Shared<N>* to = cl.map_shared_rank(sh, 0);
    if (tid == 0) to->box[rank] = s;
    if (tid < a.top) to->first[rank * a.top + tid] = sh->kept[tid];
    cl.sync();
    if (rank) return;
    s = lane < C ? sh->box[lane] : Sums();
    s.over_warp();
    if (a.top) order_list<N>(sh->first, C * a.top, sh->kept, a.top);
  }
  // (NaN and +inf: Z is NaN; no logit: Z is 0)
  const float log_z = logf(s.z), ref = s.m > -INFINITY ? s.m : 0.f;
  if (tid == 0) {
    float v = 0.f;
    if (t >= a.vocab)
      v = NAN;
    else if (t >= 0)
      v = s.z == 0.f ? -INFINITY : x_t - ref - log_z;
    a.logprobs[r] = v;
    a.entropy[r] = s.z == 0.f ? 0.f : log_z - s.u / s.z;
  }
  if (tid < a.top) {
    const uint64_t o = sh->kept[tid];
    a.top_tokens[(int64_t)r * a.top + tid] = o ? (int)(0xffffffffu - (uint32_t)o) : -1;
    a.top_logprobs[(int64_t)r * a.top + tid] = o ? of_key((uint32_t)(o >> 32)) - ref - log_z : -INFINITY;
  }
}

template <typename T, int N>
cudaError_t launch_as(const Args& a, int cluster, cudaStream_t st) {
  static_assert(sizeof(Shared<N>) <= 48 * 1024);
  return ops_launch(score_kernel<T, N>, dim3((unsigned)a.rows * cluster), N, (int)sizeof(Shared<N>), cluster, st, a);
}

template <typename T>
cudaError_t launch(const Args& a, cudaStream_t st) {
  const int granules = (int)(((int64_t)a.vocab * sizeof(T) + 15) / 16), places = 4 * ops_sm_count();
  // Many rows: with 64 KB or more 256 threads to a row, and the fewest of them have nothing to
  // do with 128 below (2048 x 131072, 20 alternatives, 93 us, with 128 threads 102; 2000 x
  // 20000 21, with 256 28).
  if (a.rows > places) return granules >= 4096 ? launch_as<T, 256>(a, 1, st) : launch_as<T, 128>(a, 1, st);
  // A row is shared among as many CTAs as leave each thread some granules and all CTAs a
  // place: four to a multiprocessor are resident.
  int C = 1;
  while (C < kMaxCluster && granules / C > 512 && (int64_t)a.rows * C * 2 <= places) C *= 2;
  return launch_as<T, 256>(a, C, st);
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
