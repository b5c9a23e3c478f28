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
// is the chain of row-wide decisions (largest logit, total weight, the prefix's
// end, the drawn token) and the arithmetic of the weights.  A cluster of CTAs
// takes one row and holds it in shared memory, so a decision costs a cluster
// barrier; a CTA leaves what the others need in their shared memory before it.
//   - Candidates.  The kept tokens are among the logits from some value up: from
//     min_p's, or from where k threads have their largest logit (each of those
//     is one of the k largest or below them).  One pass adds up the weights, if
//     p asks for the row's, and gathers the candidates; a few hundred of them
//     are ordered exactly (logit, index) and walked with exact sums by one CTA.
//   - Where they do not fit, or p keeps more than them: a histogram of the
//     distance to the largest logit, in linear bins, counts (k) or weighs (p)
//     the row.  Bins are at most 1/64 wide in y, so an element's weight is its
//     bin's upper one times 1 - z + z^2/2 to 2^-20, and one 32-bit add per
//     element does.  The bin where the rule is met is gathered, ordered and
//     walked, and a last pass draws from the row.
//   - Where that bin holds too many (flat or coarsely rounded rows), radix
//     selection on the logits' ordered bits takes over, with exact sums.
//
// One row of 5000 takes 8.4 us (k and p: some seven barriers and an ordered list),
// 64 rows of 131071 with p and min_p 30 us (0.56 TB/s: 2.5 us of reading, the
// rest the passes over shared memory and the barriers, at which the warps wait
// most), with p alone, mostly by the histogram, 66, with k alone 18, and where
// fewer logits than k are not masked, by radix selection, 81.
#include <cooperative_groups.h>

#include <type_traits>

#include "wfst_ops.h"

namespace cg = cooperative_groups;

namespace wfst {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kCoarse = kBins / 32;
constexpr int kList = 1024;          // candidates that are ordered
constexpr int kSmall = 64;           // ordered by counting all of them, from there on those of their bin
constexpr int kGuess = 192;          // threads whose largest logit p's first guess covers
constexpr int kStage = 65 * 1024;    // bytes of a row's share that are held in shared memory (64 rows of 131071: 30 us, without 32)
constexpr int kMaxCluster = 8;
constexpr int kFixed = 43;
constexpr float kMost = 3.402823466e38f;

constexpr float kHottest = 3.0e38f;  // temperature at most: its reciprocal is not zero

struct Args {
  const void* logits;
  const float *u, *temp_v, *top_p_v, *min_p_v;
  const int32_t* top_k_v;
  int32_t* token;
  float* logprob;
  int32_t* kept;
  int64_t stride;
  int32_t vocab, top_k, staged;
  float temp, top_p, min_p;
};

// NaN counts as -inf, +inf as its type's largest number (and a row that has it is
// drawn from at next to no temperature, so that no other logit weighs anything).
template <typename T>
constexpr float kLargest = kMost;
template <>
constexpr float kLargest<__half> = 65504.f;
template <>
constexpr float kLargest<__nv_bfloat16> = 3.38953138925e38f;
constexpr float kCold = 1e-36f;
template <typename T>
__device__ __forceinline__ float finite(float v) {
  return fminf(v, kLargest<T>);
}
// Larger logit, larger key; -0 and +0 have one.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
// Order of the tokens: larger logit first, then lower index.
__device__ __forceinline__ uint64_t order_of(float x, int e) {
  return (uint64_t)key_of(x) << 32 | (0xffffffffu - (uint32_t)e);
}
__device__ __forceinline__ float logit_of(uint64_t order) { return of_key((uint32_t)(order >> 32)); }
__device__ __forceinline__ int index_of(uint64_t order) { return (int)(0xffffffffu - (uint32_t)order); }

// Sums of floor(w * 2^43), 0 <= w <= 1.  Adding 8 towards zero leaves
// floor(w * 2^20) in the low mantissa bits, adding 2^-20 to the rest floor(rest *
// 2^43): two 32-bit sums of bit patterns, each pattern less its constant.  They
// hold 512 weights.
struct Fixed {
  uint32_t hi = 0, lo = 0;
  __device__ __forceinline__ void add(float w) {
    const float t = __fadd_rz(w, 8.f);
    const float rest = w - (t - 8.f);
    hi += __float_as_uint(t) - 0x41000000u;
    lo += __float_as_uint(__fadd_rz(rest, 9.5367431640625e-7f)) - 0x35800000u;
  }
  __device__ __forceinline__ uint64_t sum() const { return ((uint64_t)hi << 23) + lo; }
};
__device__ __forceinline__ uint64_t fixed_of(float w) {
  Fixed f;
  f.add(w);
  return f.sum();
}

template <typename T>
struct Row {
  static constexpr int VEC = 16 / (int)sizeof(T);
  const T* p;
  int vocab, pad;  // pad: elements between the 16-byte boundary before p and p
  // granule i: elements [i * VEC - pad, i * VEC - pad + VEC), -inf outside and for NaN
  __device__ __forceinline__ void load(int i, float (&v)[VEC]) const {
    const int e = i * VEC - pad;
    if (e >= 0 && e + VEC <= vocab) {
      const uint4 raw = *reinterpret_cast<const uint4*>(p + e);
      const T* r = reinterpret_cast<const T*>(&raw);
#pragma unroll
      for (int j = 0; j < VEC; j++) v[j] = fmaxf(to_f32(r[j]), -INFINITY);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; j++) v[j] = e + j >= 0 && e + j < vocab ? fmaxf(to_f32(p[e + j]), -INFINITY) : -INFINITY;
    }
  }
};

struct alignas(16) Shared {  // the row's granules lie behind it
  uint32_t hist[kBins];
  uint64_t list[kList];   // the candidates, gathered
  uint64_t mine[kList];   // what this CTA found
  uint64_t weight[kList], extra[kList];
  // from the cluster's CTAs, one slot each; one array per use
  uint64_t box_coarse[kMaxCluster][kCoarse], box_sum[4][kMaxCluster];
  uint32_t box_count[2][kMaxCluster];
  float box_top[kMaxCluster];
  uint64_t warp_a[kWarps], scan[kWarps + 1];
  uint32_t warp_b[kWarps];
  uint64_t cut, above;
  uint32_t bin, count, least, most;
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int x = 16; x; x /= 2) v += __shfl_xor_sync(0xffffffffu, v, x);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, v, d);
    if ((threadIdx.x & 31) >= d) v += up;
  }
  return v;
}
// Inclusive sums over the CTA's threads of one value each; *all is their total.
__device__ __forceinline__ uint64_t cta_scan(uint64_t v, Shared* sh, uint64_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v);
  __syncthreads();
  if (lane == 31) sh->scan[warp] = v;
  __syncthreads();
  uint64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    if (w < warp) before += sh->scan[w];
    total += sh->scan[w];
  }
  *all = total;
  return before + v;
}

// Descending order of list[0 .. n), n <= kList, into `to`.  bin(v) sorts no
// higher value behind a lower one: a value's place is what the bins before hold
// and what is larger in its own.  Uses sh->hist.
template <typename F>
__device__ void sort_list(const uint64_t* list, uint64_t* to, int n, Shared* sh, F bin) {
  const int tid = threadIdx.x;
  if (n <= kSmall) {
    if (tid < n) {
      const uint64_t v = list[tid];
      int r = 0;
      for (int i = 0; i < n; i++) r += list[i] > v;
      to[r] = v;
    }
    __syncthreads();
    return;
  }
  constexpr int P = kBins / kThreads, Q = kList / kThreads;
  for (int i = tid; i < kBins; i += kThreads) sh->hist[i] = 0;
  __syncthreads();
  uint32_t slot[Q];
#pragma unroll
  for (int q = 0; q < Q; q++)
    if (tid + q * kThreads < n) slot[q] = atomicAdd(&sh->hist[bin(list[tid + q * kThreads])], 1u);
  __syncthreads();
  uint32_t c[P];
  uint64_t mine = 0, all;
#pragma unroll
  for (int i = 0; i < P; i++) mine += c[i] = sh->hist[tid * P + i];
  uint32_t run = (uint32_t)(cta_scan(mine, sh, &all) - mine);
#pragma unroll
  for (int i = 0; i < P; i++) {
    sh->hist[tid * P + i] = run;  // where the bin begins
    run += c[i];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < Q; q++)
    if (tid + q * kThreads < n) {
      const uint64_t v = list[tid + q * kThreads];
      to[sh->hist[bin(v)] + slot[q]] = v;
    }
  __syncthreads();
  uint64_t v[Q];
  uint32_t r[Q];
#pragma unroll
  for (int q = 0; q < Q; q++)
    if (tid + q * kThreads < n) {
      v[q] = to[tid + q * kThreads];
      const int b = bin(v[q]);
      const uint32_t from = sh->hist[b], end = b + 1 < kBins ? sh->hist[b + 1] : (uint32_t)n;
      r[q] = from;
      for (uint32_t i = from; i < end; i++) r[q] += to[i] > v[q];
    }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < Q; q++)
    if (tid + q * kThreads < n) to[r[q]] = v[q];
  __syncthreads();
}

// One row, one cluster.  What is computed from all CTAs' values is computed by
// all CTAs alike, so that branches on it are the cluster's.
template <typename T>
struct Draw {
  static constexpr int VEC = Row<T>::VEC;
  Row<T> row;
  Shared* sh;
  uint4* stage;  // this CTA's granules, if they fit
  cg::cluster_group cl;
  int C, rank, tid, lane, warp, granules, parts, part, first, lo, hi;
  float top, inv_t, per_x;  // per_x: bins of one unit of x

  __device__ __forceinline__ float y_of(float x) const { return (x - top) * inv_t; }
  __device__ __forceinline__ float w_of(float x) const { return expf(y_of(x)); }
  // distance to the largest logit in bins, and its whole part (adding 2^23
  // towards zero leaves it in the mantissa: conversions are slow)
  __device__ __forceinline__ float far_of(float x) const { return fminf((top - x) * per_x, (float)(kBins - 1)); }
  __device__ __forceinline__ int bin_of(float x) const {
    return (int)(__float_as_uint(__fadd_rz(far_of(x), 8388608.f)) & (kBins - 1));
  }
  template <typename V>
  __device__ __forceinline__ V* at(V* p, int r) {
    return cl.map_shared_rank(p, r);
  }
  __device__ __forceinline__ void sync() {
    if (C == 1)
      __syncthreads();
    else
      cl.sync();
  }
  // Leaves a value that a whole warp has in this CTA's slot of every CTA's box.
  template <typename V>
  __device__ __forceinline__ void leave(V* box, V v) {
    if (lane < C) *at(&box[rank], lane) = v;
  }
  // The sum over all warps of all CTAs; one array of boxes per use.
  __device__ __forceinline__ uint64_t cluster_sum(uint64_t v, int use) {
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) sh->warp_a[warp] = v;
    __syncthreads();
    if (warp == 0) {
      v = warp_sum(lane < kWarps ? sh->warp_a[lane] : 0);
      leave(sh->box_sum[use], v);
    }
    sync();
    v = 0;
    for (int r = 0; r < C; r++) v += sh->box_sum[use][r];
    return v;
  }

  __device__ __forceinline__ void get(int i, float (&v)[VEC]) const {
    if (stage) {
      const uint4 raw = stage[i - first];
      const T* r = reinterpret_cast<const T*>(&raw);
#pragma unroll
      for (int j = 0; j < VEC; j++) v[j] = to_f32(r[j]);
    } else {
      row.load(i, v);
#pragma unroll
      for (int j = 0; j < VEC; j++) v[j] = finite<T>(v[j]);
    }
  }
  // f(element, logit) for each element of this warp's run of granules and for
  // the places beside the row in its first and last granule, which are -inf
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll 2
    for (int i = lo + lane; i < hi; i += 32) {
      float v[VEC];
      get(i, v);
#pragma unroll
      for (int j = 0; j < VEC; j++) f(i * VEC - row.pad + j, v[j]);
    }
  }
  // The candidates in order.  Their bins are linear in the logit's bits between
  // the list's ends, and in the index among equal ones, of which rounded logits
  // have many.
  __device__ __forceinline__ void sort(uint64_t* to, int n) {
    constexpr int kStep = std::is_same_v<T, float> ? 0 : std::is_same_v<T, __half> ? 13 : 16;  // bits without content
    uint32_t k0 = 0xffffffffu, k1 = 0;
    for (int i = tid; i < n; i += kThreads) {
      k0 = min(k0, (uint32_t)(sh->list[i] >> 32));
      k1 = max(k1, (uint32_t)(sh->list[i] >> 32));
    }
    if (tid == 0) sh->least = 0xffffffffu, sh->most = 0;
    __syncthreads();
    k0 = __reduce_min_sync(0xffffffffu, k0);
    k1 = __reduce_max_sync(0xffffffffu, k1);
    if (lane == 0 && k0 <= k1) {
      atomicMin(&sh->least, k0);
      atomicMax(&sh->most, k1);
    }
    __syncthreads();
    const uint32_t last = sh->most;
    const float scale = (float)kBins / ((float)((last - sh->least) >> kStep) + 1.f), per = 1.f / (float)row.vocab;
    sort_list(sh->list, to, n, sh, [&](uint64_t v) {
      const float at = (float)((last - (uint32_t)(v >> 32)) >> kStep) + fminf((float)index_of(v) * per, 1.f);
      return min((int)(at * scale), kBins - 1);
    });
  }
  __device__ __forceinline__ bool in_row(int e) const { return e >= 0 && e < row.vocab; }

  // The bin where the running sum over all CTAs' histograms reaches `want`;
  // *above: the sum before it.  Bins count as value(bin, sum).  kBins if it is
  // never reached.  The histogram must stay until the next cluster barrier.  COUNT:
  // value is the sum itself.
  template <bool COUNT, typename F>
  __device__ int find_bin(uint64_t want, uint64_t* above, F value) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCoarse / kWarps; i++) {
      const int c = warp * (kCoarse / kWarps) + i;
      uint64_t v;
      if constexpr (COUNT)
        v = __reduce_add_sync(0xffffffffu, sh->hist[c * 32 + lane]);
      else
        v = warp_sum(value(c * 32 + lane, sh->hist[c * 32 + lane]));
      if (lane < C) at(&sh->box_coarse[rank][0], lane)[c] = v;
    }
    sync();
    // every warp the same
    uint64_t v0 = 0, v1 = 0;
    for (int r = 0; r < C; r++) {
      v0 += sh->box_coarse[r][2 * lane];
      v1 += sh->box_coarse[r][2 * lane + 1];
    }
    uint64_t run = warp_scan(v0 + v1) - (v0 + v1);
    const bool here = run < want && want <= run + v0 + v1;
    const unsigned who = __ballot_sync(0xffffffffu, here);
    if (!who) return kBins;
    const bool second = want > run + v0;
    const int c = __shfl_sync(0xffffffffu, 2 * lane + (second ? 1 : 0), __ffs(who) - 1);
    const uint64_t before = __shfl_sync(0xffffffffu, second ? run + v0 : run, __ffs(who) - 1);
    const int b = c * 32 + lane;
    uint64_t v = 0;
    for (int r = 0; r < C; r++) v += value(b, *at(&sh->hist[b], r));
    run = before + warp_scan(v) - v;
    const unsigned at_bin = __ballot_sync(0xffffffffu, run < want && want <= run + v);
    if (!at_bin) return kBins;  // (weights: their parts may round otherwise than their sum)
    *above = __shfl_sync(0xffffffffu, run, __ffs(at_bin) - 1);
    return __shfl_sync(0xffffffffu, b, __ffs(at_bin) - 1);
  }

  __device__ void clear_hist() {
    for (int i = tid; i < kBins; i += kThreads) sh->hist[i] = 0;
    if (tid == 0) sh->count = 0;
    __syncthreads();
  }

  __device__ __forceinline__ void put(uint64_t v) {
    const uint32_t i = atomicAdd(&sh->count, 1u);
    if (i < (uint32_t)kList) sh->mine[i] = v;
  }
  // How many tokens the CTAs have put into their `mine`, -1 if they do not fit
  // one list.  Gathers them in `list`, in every CTA or the first one.
  __device__ int gather(bool everywhere, int use) {
    __syncthreads();
    if (warp == 0) leave(sh->box_count[use], sh->count);
    sync();
    int n = 0;
    for (int r = 0; r < C; r++) n += (int)min(sh->box_count[use][r], (uint32_t)kList + 1);
    if (n > kList) return -1;
    if (!everywhere && rank) return n;
    int from = 0;
    for (int r = 0; r < C; r++) {
      const int c = (int)sh->box_count[use][r];
      const uint64_t* src = at(&sh->mine[0], r);
      for (int i = tid; i < c; i += kThreads) sh->list[from + i] = src[i];
      from += c;
    }
    __syncthreads();
    return n;
  }

  // Radix selection over the tokens at or before `cut`: the order of the last
  // one of the shortest prefix that reaches `want` tokens (or weight).
  __device__ uint64_t select_slow(bool by_weight, uint64_t want, uint64_t cut) {
    uint32_t prefix = 0, mask = 0;
    constexpr int P = kBins / kThreads;
    for (int level = 0; level < 3; level++) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
      const uint32_t width = level == 2 ? 0x3ffu : 0x7ffu;
      // a weight is three pieces of 15 bits, whose sums over a CTA's share of a
      // row stay below 2^32: one histogram after the other
      uint64_t sum[P] = {};
      for (int piece = 0; piece < (by_weight ? 3 : 1); piece++) {
        sync();
        clear_hist();
        each([&](int e, float x) {
          const uint32_t key = key_of(x);
          if ((key & mask) != prefix || !in_row(e) || order_of(x, e) < cut) return;
          const uint32_t v = by_weight ? (uint32_t)(fixed_of(w_of(x)) >> (15 * piece)) & 0x7fffu : 1u;
          if (v) atomicAdd(&sh->hist[key >> shift & width], v);
        });
        sync();
#pragma unroll
        for (int i = 0; i < P; i++)
          for (int r = 0; r < C; r++) sum[i] += (uint64_t)*at(&sh->hist[kBins - 1 - (tid * P + i)], r) << (15 * piece);
      }
      uint64_t mine = 0, all;
#pragma unroll
      for (int i = 0; i < P; i++) mine += sum[i];
      uint64_t run = cta_scan(mine, sh, &all) - mine;
#pragma unroll
      for (int i = 0; i < P; i++) {
        if (run < want && want <= run + sum[i]) {
          sh->bin = kBins - 1 - (tid * P + i);
          sh->above = run;
        }
        run += sum[i];
      }
      __syncthreads();
      want -= sh->above;
      prefix |= sh->bin << shift;
      mask |= width << shift;
    }
    // equal logits: the n-th of them by index
    uint64_t n = want;
    if (by_weight) {
      const uint64_t w = fixed_of(w_of(of_key(prefix)));
      n = (want + w - 1) / w;
    }
    uint32_t c = 0;
    each([&](int e, float x) { c += key_of(x) == prefix && in_row(e) && order_of(x, e) >= cut; });
    const uint32_t here = (uint32_t)warp_sum(c);
    if (lane == 0) sh->warp_b[warp] = here;
    sync();
    uint64_t before = 0;
    for (int i = 0; i < part; i++) before += *at(&sh->warp_b[i % kWarps], i / kWarps);
    if (before < n && n <= before + here) {  // this warp's run holds it
      uint64_t left = n - before;
      for (int i0 = lo; i0 < hi; i0 += 32) {
        float v[VEC] = {};
        uint32_t mine = 0;
        auto counts = [&](int j) {
          const int e = (i0 + lane) * VEC - row.pad + j;
          return key_of(v[j]) == prefix && in_row(e) && order_of(v[j], e) >= cut;
        };
        if (i0 + lane < hi) {
          get(i0 + lane, v);
#pragma unroll
          for (int j = 0; j < VEC; j++) mine += counts(j);
        }
        const uint32_t incl = (uint32_t)warp_scan(mine);
        const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
        if (left > all) {
          left -= all;
          continue;
        }
        if (incl >= left && incl - mine < left) {
          uint32_t k = incl - mine;
#pragma unroll
          for (int j = 0; j < VEC; j++)
            if (counts(j) && ++k == left)
              for (int r = 0; r < C; r++) *at(&sh->cut, r) = order_of(v[j], (i0 + lane) * VEC - row.pad + j);
        }
        break;
      }
    }
    sync();
    return sh->cut;
  }

  // An element's weight as a share of its bin's upper one, in units of 2^-17.
  __device__ __forceinline__ uint32_t share_of(float x) const {
    const float d = far_of(x);
    const float z = (d - (__fadd_rz(d, 8388608.f) - 8388608.f)) * (inv_t / per_x);
    const float share = __fmaf_rn(__fmaf_rn(65536.f, z, -131072.f), z, 131072.5f);
    return __float_as_uint(__fadd_rz(share, 8388608.f)) & 0x3ffffu;
  }

  // The same as select_slow's through the histogram of distances.  *kept: this
  // warp's share of the prefix, where `sums` says that it is known (for weights).
  __device__ uint64_t select(bool by_weight, uint64_t want, uint64_t cut, uint64_t* kept_w, uint32_t* kept_c, bool* sums) {
    *sums = false;
    sync();
    clear_hist();
    const float x_first = logit_of(cut);
    auto at_or_before = [&](int e, float x) { return !cut || x > x_first || (x == x_first && order_of(x, e) >= cut); };
    each([&](int e, float x) {
      if (at_or_before(e, x)) atomicAdd(&sh->hist[bin_of(x)], by_weight ? share_of(x) : 1u);
    });
    uint64_t above = 0;
    const float width = inv_t / per_x;  // of a bin, in y
    const int bin =
        by_weight ? find_bin<false>(want, &above,
                                    [&](int b, uint32_t sum) {
                                      return (uint64_t)((float)sum * expf(-width * b) * (float)(1 << (kFixed - 17)));
                                    })
                  : find_bin<true>(want, &above, [](int, uint32_t sum) { return (uint64_t)sum; });
    if (bin < kBins - 1) {  // (the last bin has no lower end)
      Fixed f;
      uint32_t c = 0;
      each([&](int e, float x) {
        const float far = far_of(x);
        if (far >= (float)(bin + 1) || !at_or_before(e, x)) return;
        if (far >= (float)bin) {
          put(order_of(x, e));
        } else if (by_weight) {
          f.add(w_of(x));
          c++;
        }
      });
      *kept_w = warp_sum(f.sum());
      *kept_c = __reduce_add_sync(0xffffffffu, c);
      if (by_weight) above = cluster_sum(f.sum(), 2 + (cut != 0));
      const int n = gather(true, cut != 0);
      if (n >= 0 && above < want) {
        uint64_t* order = sh->weight;
        sort(order, n);
        constexpr int P = kList / kThreads;
        uint64_t v[P], mine = 0, all;
#pragma unroll
        for (int i = 0; i < P; i++) {
          const int k = tid * P + i;
          v[i] = k >= n ? 0 : by_weight ? fixed_of(w_of(logit_of(order[k]))) : 1;
          mine += v[i];
        }
        uint64_t run = above + cta_scan(mine, sh, &all) - mine;
        if (above + all >= want) {
#pragma unroll
          for (int i = 0; i < P; i++) {
            if (run < want && want <= run + v[i]) sh->cut = order[tid * P + i];
            run += v[i];
          }
          __syncthreads();
          const uint64_t end = sh->cut;
          // those of the bin that are in this warp's run of the row
          const int e0 = lo * VEC - row.pad, e1 = hi * VEC - row.pad;
          Fixed g;
          c = 0;
          for (int i = lane; i < n; i += 32) {
            const int e = index_of(order[i]);
            if (order[i] >= end && e >= e0 && e < e1) {
              g.add(w_of(logit_of(order[i])));
              c++;
            }
          }
          *kept_w += warp_sum(g.sum());
          *kept_c += __reduce_add_sync(0xffffffffu, c);
          *sums = by_weight;
          return end;
        }
      }
    }
    return select_slow(by_weight, want, cut);
  }
};

__device__ __forceinline__ uint64_t goal_of(float p, uint64_t sum) {
  const double goal = ceil((double)sum * (double)p);
  const uint64_t want = goal >= 1.0 ? (uint64_t)goal : 1;
  return want < sum ? want : sum;
}
__device__ __forceinline__ uint64_t aim_of(float u, uint64_t total) {
  const double goal = (double)u * (double)total;
  const uint64_t aim = goal > 0.0 ? (uint64_t)goal : 0;
  return aim < total - 1 ? aim : total - 1;
}
__device__ __forceinline__ float logprob_of(float y, uint64_t total) {
  return y - logf((float)total * (1.f / (1ull << kFixed)));
}

static_assert(sizeof(Shared) % 16 == 0);

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char raw_smem[];
  Draw<T> d{{}, reinterpret_cast<Shared*>(raw_smem), nullptr, cg::this_cluster()};
  Shared* sh = d.sh;
  const int C = d.C = (int)d.cl.num_blocks(), rank = d.rank = (int)d.cl.block_rank();
  // A CTA's shared memory may be written by the others once it runs: that all of
  // them do is known at the wait before the first `leave`, behind the row's reading.
  if (C > 1) d.cl.barrier_arrive();
  ops_begin();
  ops_next();
  const int b = blockIdx.x / C;
  const int tid = d.tid = threadIdx.x, lane = d.lane = tid & 31, warp = d.warp = tid >> 5;
  constexpr int VEC = Row<T>::VEC;
  d.row.p = reinterpret_cast<const T*>(a.logits) + b * a.stride;
  d.row.vocab = a.vocab;
  d.row.pad = (int)(((uintptr_t)d.row.p & 15) / sizeof(T));
  d.granules = (a.vocab + d.row.pad + VEC - 1) / VEC;
  // each warp of the cluster has a run of granules, in index order
  const int parts = d.parts = C * kWarps, part = d.part = rank * kWarps + warp;
  d.lo = (int)((int64_t)d.granules * part / parts), d.hi = (int)((int64_t)d.granules * (part + 1) / parts);
  d.first = (int)((int64_t)d.granules * rank / C);

  float temp = a.temp_v ? a.temp_v[b] : a.temp;
  int k = a.top_k_v ? a.top_k_v[b] : a.top_k;
  const float top_p = a.top_p_v ? a.top_p_v[b] : a.top_p;
  const float min_p = fminf(a.min_p_v ? a.min_p_v[b] : a.min_p, 1.f);
  const float u = a.u[b];
  if (!(temp > 0.f)) {
    temp = 1.f;
    k = 1;
  }
  temp = fminf(temp, kHottest);
  const bool by_k = k > 0 && k < a.vocab, by_p = top_p < 1.f || top_p != top_p, by_min = min_p > 0.f;

  // ---- the largest logit; the row comes into shared memory
  float most = -INFINITY;  // this thread's
  uint4* stage = a.staged ? reinterpret_cast<uint4*>(raw_smem + sizeof(Shared)) : nullptr;
#pragma unroll 4
  for (int i = d.lo + lane; i < d.hi; i += 32) {
    float v[VEC];
    d.row.load(i, v);
    uint4 raw;
    T* r = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      r[j] = from_f32<T>(finite<T>(v[j]));
      most = fmaxf(most, v[j]);
    }
    if (stage) stage[i - d.first] = raw;  // read back by this lane alone
  }
  d.stage = stage;
  d.clear_hist();
  float top = most;
#pragma unroll
  for (int x = 16; x; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  if (lane == 0) sh->warp_b[warp] = __float_as_uint(top);
  __syncthreads();
  if (C > 1) d.cl.barrier_wait();  // all CTAs of the cluster run
  if (warp == 0) {
    top = lane < kWarps ? __uint_as_float(sh->warp_b[lane]) : -INFINITY;
#pragma unroll
    for (int x = 16; x; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    d.leave(sh->box_top, top);
  }
  d.sync();
  top = sh->box_top[0];
  for (int r = 1; r < C; r++) top = fmaxf(top, sh->box_top[r]);
  if (top == INFINITY) temp = kCold;
  d.top = top = finite<T>(top);
  most = finite<T>(most);
  d.inv_t = fminf(1.f / temp, kMost);
  // the bins reach 32 in y, past which nothing weighs anything, or 24 in x
  d.per_x = fminf((float)kBins / fminf(32.f * temp, 24.f), kMost);
  if (top == -INFINITY) {  // nothing to draw from
    if (rank == 0 && tid == 0) {
      a.token[b] = -1;
      a.logprob[b] = -INFINITY;
      a.kept[b] = 0;
    }
    d.sync();
    return;
  }

  // ---- the candidates: logits from x_c up, all kept ones among them
  float x_c = -INFINITY;
  if (by_k || (by_p && !by_min)) {
    const int need = by_k ? k : kGuess;
    if (need <= C * kThreads) {
      if (most > -INFINITY) atomicAdd(&sh->hist[d.bin_of(most)], 1u);
      uint64_t above;
      const int bin = d.template find_bin<true>((uint64_t)need, &above, [](int, uint32_t sum) { return (uint64_t)sum; });
      // at or below the bin's lower end
      if (bin < kBins - 1) x_c = __fadd_rd(top, -(bin + 1) / d.per_x * 1.00001f);
    }
  }
  // at or below the last logit whose weight is min_p (but p's share is of all k)
  if (by_min && !(by_k && by_p)) x_c = fmaxf(x_c, __fadd_rd(top, (logf(min_p) * 1.0001f - 0.001f) * temp));
  const bool some = x_c > -INFINITY, all_weights = by_p && !by_k;
  uint64_t total = 0, cut = 0;
  int n = -1;
  bool sums = false;  // this warp's share of the kept tokens is known:
  uint64_t mine = 0;
  uint32_t mine_c = 0;
  if (some || all_weights) {
    Fixed f, g;  // of all logits, of those that min_p keeps
    uint32_t c = 0;
    const bool apart = by_min && !by_k;
    d.each([&](int e, float x) {
      if (all_weights) f.add(d.w_of(x));
      if (some && x >= x_c) {
        d.put(order_of(x, e));
        if (apart) {
          const float w = d.w_of(x);
          if (w >= min_p) {
            g.add(w);
            c++;
          }
        }
      }
    });
    if (all_weights) total = d.cluster_sum(f.sum(), 0);
    if (some) n = d.gather(false, 0);
    if (n < 0 && apart) {  // too many for the list; min_p may end the prefix before p does
      mine = warp_sum(g.sum());
      mine_c = __reduce_add_sync(0xffffffffu, c);
      sums = !by_p || d.cluster_sum(g.sum(), 1) < goal_of(top_p, total);
    }
  }
  if (n >= 0) {
    // ---- the first CTA decides on the list
    if (rank == 0) {
      uint64_t* order = sh->mine;
      d.sort(order, n);
      constexpr int P = kList / kThreads;
      const int m0 = by_k && k < n ? k : n;
      uint64_t v[P], part_sum = 0, all;
      float w[P];
#pragma unroll
      for (int i = 0; i < P; i++) {
        const int j = tid * P + i;
        w[i] = j < m0 ? d.w_of(logit_of(order[j])) : 0.f;
        v[i] = j < m0 ? fixed_of(w[i]) : 0;
        if (j < n) sh->weight[j] = v[i];
        part_sum += v[i];
      }
      uint64_t run = cta_scan(part_sum, sh, &all) - part_sum;
      uint64_t want = UINT64_MAX;
      if (by_p) {  // in one warp: 64-bit floating point is slow here
        if (warp == 0) sh->above = goal_of(top_p, by_k ? all : total);
        __syncthreads();
        want = sh->above;
      }
      // (what min_p or k ends needs no more than the candidates)
      const bool enough = by_k || by_min || all >= want;
      int c = 0;
#pragma unroll
      for (int i = 0; i < P; i++) {
        c += tid * P + i < m0 && run < want && w[i] >= min_p;
        run += v[i];
      }
      // the kept ones are a prefix: threads with all of theirs, one with some
      const int m = __syncthreads_count(c == P) * P + __syncthreads_count(c == 1);
      static_assert(P == 2, "a thread keeps none, one or two");
      if (!enough) {
        n = -1;
      } else {
        auto answer = [&](uint64_t it, uint64_t sum) {
          a.token[b] = index_of(it);
          a.logprob[b] = logprob_of(d.y_of(logit_of(it)), sum);
          a.kept[b] = m;
        };
        if (m <= kThreads / 4) {
          // each kept token's place in the cumulative weight in index order, by
          // counting; four lanes share a token
          const int i = tid / 4;
          if (warp * 8 < m) {
            uint64_t before = 0, sum = 0;
            const uint32_t own = i < m ? (uint32_t)order[i] : 0;
            for (int j = tid % 4; j < m; j += 4) {
              const uint64_t f = sh->weight[j];
              sum += f;
              if ((uint32_t)order[j] > own) before += f;  // a lower index
            }
            for (int x = 1; x < 4; x *= 2) {
              sum += __shfl_xor_sync(0xffffffffu, sum, x);
              before += __shfl_xor_sync(0xffffffffu, before, x);
            }
            const uint64_t aim = aim_of(u, sum);
            if (i < m && tid % 4 == 0 && before <= aim && aim < before + sh->weight[i]) answer(order[i], sum);
          }
        } else {
          // ordered by index, each with its place in the order of logits
          for (int i = tid; i < m; i += kThreads) sh->list[i] = (order[i] & 0xffffffffull) << 32 | (uint32_t)i;
          __syncthreads();
          const float per = (float)kBins / (float)a.vocab;
          sort_list(sh->list, sh->extra, m, sh, [&](uint64_t v) {
            return min((int)((float)(0xffffffffu - (uint32_t)(v >> 32)) * per), kBins - 1);
          });
          part_sum = 0;
#pragma unroll
          for (int i = 0; i < P; i++) {
            const int j = tid * P + i;
            v[i] = j < m ? sh->weight[(uint32_t)sh->extra[j]] : 0;
            part_sum += v[i];
          }
          run = cta_scan(part_sum, sh, &all) - part_sum;
          if (warp == 0) sh->above = aim_of(u, all);
          __syncthreads();
          const uint64_t aim = sh->above;
#pragma unroll
          for (int i = 0; i < P; i++) {
            if (run <= aim && aim < run + v[i]) answer(order[(uint32_t)sh->extra[tid * P + i]], all);
            run += v[i];
          }
        }
      }
    }
    if (all_weights && !by_min) {  // the guess for p may have been too small
      if (warp == 0 && rank == 0 && lane < C) *d.at(&sh->bin, lane) = n >= 0;
      d.sync();
      n = sh->bin ? 0 : -1;
    } else {
      d.sync();  // no CTA leaves while another may read its shared memory
    }
    if (n >= 0) return;
  }

  // ---- the end of the kept prefix in the whole row
  if (!sums) {
    if (by_k) {
      cut = d.select(false, (uint64_t)k, 0, &mine, &mine_c, &sums);
      if (by_p) {
        Fixed f;
        d.each([&](int e, float x) {
          if (order_of(x, e) >= cut) f.add(d.w_of(x));
        });
        total = d.cluster_sum(f.sum(), 0);
      }
    }
    if (by_p) cut = d.select(true, goal_of(top_p, total), cut, &mine, &mine_c, &sums);
    sums = sums && !by_min;
  }

  // ---- the draw: kept are the tokens of at least this order, and of min_p's weight
  const float x_cut = cut ? logit_of(cut) : -INFINITY;
  auto weigh = [&](int e, float x, float* w) {
    if (x < x_cut || (cut && order_of(x, e) < cut)) return false;
    *w = d.w_of(x);
    return *w >= min_p && d.in_row(e);
  };
  if (!sums) {
    Fixed f;
    uint32_t c = 0;
    d.each([&](int e, float x) {
      float w;
      if (weigh(e, x, &w)) {
        f.add(w);
        c++;
      }
    });
    mine = warp_sum(f.sum());
    mine_c = __reduce_add_sync(0xffffffffu, c);
  }
  d.sync();  // the boxes are free
  if (lane == 0) {
    sh->warp_a[warp] = mine;
    sh->warp_b[warp] = mine_c;
  }
  __syncthreads();
  uint64_t before = 0;  // of this CTA's warps before this one
  if (warp == 0) {
    d.leave(sh->box_sum[1], warp_sum(lane < kWarps ? sh->warp_a[lane] : 0));
    d.leave(sh->box_count[1], (uint32_t)warp_sum(lane < kWarps ? sh->warp_b[lane] : 0));
  }
  d.sync();
  uint32_t kept = 0;
  total = 0;
  for (int r = 0; r < C; r++) {
    if (r == rank) before = total;
    total += sh->box_sum[1][r];
    kept += sh->box_count[1][r];
  }
  for (int w = 0; w < warp; w++) before += sh->warp_a[w];
  const uint64_t aim = aim_of(u, total);
  if (before <= aim && aim < before + mine) {
    // the first element of this warp's run whose running sum exceeds it
    uint64_t left = aim - before;
    for (int i0 = d.lo; i0 < d.hi; i0 += 32) {
      const int i = i0 + lane;
      float x[VEC];
      uint64_t v[VEC], own = 0;
      if (i < d.hi) {
        d.get(i, x);
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          float w;
          v[j] = weigh(i * VEC - d.row.pad + j, x[j], &w) ? fixed_of(w) : 0;
          own += v[j];
        }
      }
      const uint64_t incl = warp_scan(own);
      const uint64_t all = __shfl_sync(0xffffffffu, incl, 31);
      if (all <= left) {
        left -= all;
        continue;
      }
      if (incl > left && incl - own <= left) {
        uint64_t run = incl - own;
        bool done = false;
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          run += v[j];
          if (!done && run > left) {
            done = true;
            a.token[b] = i * VEC - d.row.pad + j;
            a.logprob[b] = logprob_of(d.y_of(x[j]), total);
            a.kept[b] = (int32_t)kept;
          }
        }
      }
      break;
    }
  }
  if (C > 1) d.cl.sync();  // no CTA leaves while another may read its shared memory
}

template <typename T>
cudaError_t launch(Args& a, int lanes, cudaStream_t st) {
  // a row is split until a CTA has 8192 logits, or the CTAs fill the device (two
  // to a multiprocessor); a CTA's share stays below 2^17 logits (select_slow).
  // One row of 5000, which stays whole, takes 8.3 us, split in two 9.6; 64 rows of
  // 131071, split in four, 30, in eight 38
  int c = 1;
  while (c < kMaxCluster &&
         (a.vocab > (1 << 17) * c || (a.vocab > 8192 * c && (int64_t)lanes * c <= ops_sm_count())))
    c *= 2;
  const int share = ((a.vocab + 16) * (int)sizeof(T) / c / 16 + 2) * 16;  // bytes, at most
  a.staged = share <= kStage;
  const int smem = (int)sizeof(Shared) + (a.staged ? share : 0);
  static OpsOnce once;
  if (const int dev = ops_current(); !once(dev)) {
    const cudaError_t e =
        cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(Shared) + kStage);
    if (e != cudaSuccess) return e;
    once.set(dev);
  }
  return ops_launch(sample_kernel<T>, (unsigned)lanes * c, kThreads, smem, c, st, a);
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
  if (!r->temperature_v && !(r->temperature >= 0.f && r->temperature <= kHottest))
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
  const int dev = ops_device(r->device, {r->logits, r->uniform, r->temperature_v, r->top_k_v, r->top_p_v, r->min_p_v, r->tokens,
                              r->logprobs, r->kept});
  if (dev < 0) return api_fail(WFST_ERR_INVALID_ARG, "sample_tokens: every array must be device memory of one device");
  OpsDevice guard(dev);
  if (guard.err != cudaSuccess) return api_cuda_fail(guard.err, "sample_tokens: device");
  Args a;
  a.logits = r->logits, a.u = r->uniform;
  a.temp_v = r->temperature_v, a.top_k_v = r->top_k_v, a.top_p_v = r->top_p_v, a.min_p_v = r->min_p_v;
  a.token = r->tokens, a.logprob = r->logprobs, a.kept = r->kept;
  a.stride = r->lanes > 1 ? r->stride : 0, a.vocab = r->vocab;
  a.temp = r->temperature, a.top_k = r->top_k, a.top_p = r->top_p, a.min_p = r->min_p;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = r->dtype == WFST_F32   ? launch<float>(a, r->lanes, st)
                        : r->dtype == WFST_F16 ? launch<__half>(a, r->lanes, st)
                                               : launch<__nv_bfloat16>(a, r->lanes, st);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "sample_tokens launch");
}
