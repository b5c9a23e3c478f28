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
// decision costs a cluster barrier and not a launch.  No sort of the row:
//   - a histogram of the distance to the largest logit, in linear bins, counts
//     (k) or weighs (p) the row and tells the bin where the rule is met.  Bins
//     are at most 1/64 wide in y, so an element's weight is its bin's upper one
//     times 1 - z + z^2/2 to 2^-20, and one 32-bit add per element does;
//   - the elements of that bin are gathered, ordered exactly (logit, index) and
//     walked with exact sums;
//   - where the bin holds too many (flat or coarsely rounded rows), radix
//     selection on the logits' ordered bits takes over, with exact sums.
#include <cooperative_groups.h>

#include "wfst_ops.h"

namespace cg = cooperative_groups;

namespace wfst {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 2048;
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
};

struct Shared {
  uint32_t hist[kBins];
  uint64_t list[kList];           // every CTA's copy of what was gathered
  uint64_t mine[kList];           // what this CTA gathered
  uint64_t warp_a[4][kWarps];     // one row per use: a reader is never overtaken
  uint32_t warp_b[2][kWarps];
  float top[kWarps];
  uint64_t scan[kWarps + 1];
  uint64_t above, cut;
  uint32_t bin, count, fits;
};

// Order of the tokens: larger logit first, then lower index.
__device__ __forceinline__ uint64_t order_of(float x, int e) {
  return (uint64_t)key_of(x) << 32 | (0xffffffffu - (uint32_t)e);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int x = 16; x; x /= 2) v += __shfl_xor_sync(0xffffffffu, v, x);
  return v;
}

// Inclusive sums over the CTA's threads of one value each; *all is their total.
__device__ __forceinline__ uint64_t cta_scan(uint64_t v, Shared* sh, uint64_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += up;
  }
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

// Descending order of list[0 .. n), n <= kList (bitonic, padded with zeros).
__device__ void sort_list(uint64_t* list, int n) {
  int p = 2;
  while (p < n) p *= 2;
  for (int i = threadIdx.x; i < p; i += kThreads)
    if (i >= n) list[i] = 0;
  for (int k = 2; k <= p; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      __syncthreads();
      for (int t = threadIdx.x; t < p / 2; t += kThreads) {
        const int lo = 2 * t - (t & (j - 1)), hi = lo + j;
        const uint64_t a = list[lo], b = list[hi];
        if ((a < b) == ((lo & k) == 0)) {
          list[lo] = b;
          list[hi] = a;
        }
      }
    }
  __syncthreads();
}

// One row, one cluster.
template <typename T>
struct Draw {
  static constexpr int VEC = Row<T>::VEC;
  Row<T> row;
  Shared* sh;
  cg::cluster_group cl;
  int C, rank, tid, lane, warp, granules, parts, part, lo, hi;
  float top, inv_t, per_x;  // per_x: bins of one unit of x

  __device__ __forceinline__ float y_of(float x) const { return x == top ? 0.f : (x - top) * inv_t; }
  __device__ __forceinline__ float w_of(float x) const { return expf(y_of(x)); }
  __device__ __forceinline__ uint64_t f_of(float x) const { return fixed_of(w_of(x)); }
  __device__ __forceinline__ int bin_of(float x) const {
    return x == top ? 0 : (int)fminf((top - x) * per_x, (float)(kBins - 1));
  }
  template <typename V>
  __device__ __forceinline__ V* at(V* p, int r) {
    return cl.map_shared_rank(p, r);
  }

  // f(element, logit) for each element of this warp's run of granules
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll 2
    for (int i = lo + lane; i < hi; i += 32) {
      float v[VEC];
      row.load(i, v);
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const int e = i * VEC - row.pad + j;
        if (e >= 0 && e < row.vocab) f(e, v[j]);
      }
    }
  }

  // Sum over the cluster of one value per warp; `use` names the row of warp_a.
  __device__ __forceinline__ uint64_t cluster_sum(uint64_t v, int use) {
    v = warp_sum(v);
    if (lane == 0) sh->warp_a[use][warp] = v;
    cl.sync();
    uint64_t sum = 0;
    for (int i = lane; i < parts; i += 32) sum += *at(&sh->warp_a[use][i % kWarps], i / kWarps);
    return warp_sum(sum);
  }

  // The bin where the running sum over all CTAs' histograms, from bin 0 on (or
  // from the last one down), reaches `want`; *above: the sum before it.  Bins
  // count as value(bin, sum).  kBins if it is never reached.
  template <typename F>
  __device__ uint32_t find_bin(bool down, uint64_t want, uint64_t* above, F value) {
    constexpr int P = kBins / kThreads;
    uint64_t v[P], mine = 0;
#pragma unroll
    for (int i = 0; i < P; i++) {
      const int k = tid * P + i, b = down ? kBins - 1 - k : k;
      uint64_t sum = 0;
      for (int r = 0; r < C; r++) sum += *at(&sh->hist[b], r);
      v[i] = value(b, sum);
      mine += v[i];
    }
    uint64_t all;
    uint64_t run = cta_scan(mine, sh, &all) - mine;
    if (tid == 0) sh->bin = kBins;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < P; i++) {
      if (run < want && want <= run + v[i]) {
        sh->bin = down ? kBins - 1 - (tid * P + i) : tid * P + i;
        sh->above = run;
      }
      run += v[i];
    }
    __syncthreads();
    *above = sh->above;
    return sh->bin;
  }

  __device__ void clear_hist() {
    for (int i = tid; i < kBins; i += kThreads) sh->hist[i] = 0;
    if (tid == 0) sh->count = 0;
    __syncthreads();
  }

  // How many tokens the CTAs have put into their `mine`, -1 if they do not fit
  // one list.  Gathers and orders them in `list`, in every CTA or the first one.
  __device__ int gather(bool everywhere) {
    cl.sync();
    int n = 0, first = 0;
    bool fits = true;
    for (int r = 0; r < C; r++) {
      const int c = (int)*at(&sh->count, r);
      fits = fits && c <= kList;
      n += c;
    }
    if (!fits || n > kList) return -1;
    if (!everywhere && rank) return n;
    for (int r = 0; r < C; r++) {
      const int c = (int)*at(&sh->count, r);
      const uint64_t* from = at(&sh->mine[0], r);
      for (int i = tid; i < c; i += kThreads) sh->list[first + i] = from[i];
      first += c;
    }
    __syncthreads();
    sort_list(sh->list, n);
    return n;
  }
  __device__ __forceinline__ void put(uint64_t v) {
    const uint32_t i = atomicAdd(&sh->count, 1u);
    if (i < (uint32_t)kList) sh->mine[i] = v;
  }

  // Radix selection over the tokens at or before `cut`: the order of the last
  // one of the shortest prefix that reaches `want` tokens (or weight).
  __device__ uint64_t select_slow(bool by_weight, uint64_t want, uint64_t cut) {
    uint32_t prefix = 0, mask = 0;
    for (int level = 0; level < 3; level++) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
      const uint32_t width = level == 2 ? 0x3ffu : 0x7ffu;
      // a weight is three pieces of 15 bits, whose sums over a CTA's share of a
      // row stay below 2^32: one histogram after the other
      uint64_t sum[kBins / kThreads] = {};
      for (int piece = 0; piece < (by_weight ? 3 : 1); piece++) {
        cl.sync();
        clear_hist();
        each([&](int e, float x) {
          const uint32_t key = key_of(x);
          if ((key & mask) != prefix || order_of(x, e) < cut) return;
          const uint32_t v = by_weight ? (uint32_t)(f_of(x) >> (15 * piece)) & 0x7fffu : 1u;
          if (v) atomicAdd(&sh->hist[key >> shift & width], v);
        });
        cl.sync();
#pragma unroll
        for (int i = 0; i < kBins / kThreads; i++) {
          const int b = kBins - 1 - (tid * (kBins / kThreads) + i);
          for (int r = 0; r < C; r++) sum[i] += (uint64_t)*at(&sh->hist[b], r) << (15 * piece);
        }
      }
      uint64_t mine = 0, all;
#pragma unroll
      for (int i = 0; i < kBins / kThreads; i++) mine += sum[i];
      uint64_t run = cta_scan(mine, sh, &all) - mine;
#pragma unroll
      for (int i = 0; i < kBins / kThreads; i++) {
        if (run < want && want <= run + sum[i]) {
          sh->bin = kBins - 1 - (tid * (kBins / kThreads) + i);
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
      const uint64_t w = f_of(of_key(prefix));
      n = (want + w - 1) / w;
    }
    uint32_t c = 0;
    each([&](int e, float x) { c += key_of(x) == prefix && order_of(x, e) >= cut; });
    const uint64_t here = warp_sum(c);
    if (lane == 0) sh->warp_b[1][warp] = (uint32_t)here;
    cl.sync();
    uint64_t before = 0;
    for (int i = 0; i < parts; i++) {
      const uint64_t w = *at(&sh->warp_b[1][i % kWarps], i / kWarps);
      if (before < n && n <= before + w && i == part) {  // this warp's run holds it
        uint64_t left = n - before;
        for (int i0 = lo; i0 < hi; i0 += 32) {
          float v[VEC];
          uint32_t mine = 0;
          if (i0 + lane < hi) {
            row.load(i0 + lane, v);
#pragma unroll
            for (int j = 0; j < VEC; j++) {
              const int e = (i0 + lane) * VEC - row.pad + j;
              mine += e >= 0 && e < row.vocab && key_of(v[j]) == prefix && order_of(v[j], e) >= cut;
            }
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
          if (incl >= left && incl - mine < left) {
            uint32_t k = incl - mine;
#pragma unroll
            for (int j = 0; j < VEC; j++) {
              const int e = (i0 + lane) * VEC - row.pad + j;
              if (e >= 0 && e < row.vocab && key_of(v[j]) == prefix && order_of(v[j], e) >= cut && ++k == left)
                for (int r = 0; r < C; r++) *at(&sh->cut, r) = order_of(v[j], e);
            }
          }
          break;
        }
      }
      before += w;
    }
    cl.sync();
    return sh->cut;
  }

  // The same through the histogram of distances; `want` and the rule as there.
  // *n: where k tokens and all before them were gathered, how many lie in
  // `list` (the rest of the work happens there), else -1.
  __device__ uint64_t select(bool by_weight, uint64_t want, uint64_t cut, bool filled, int* n) {
    *n = -1;
    if (!filled) {
      each([&](int e, float x) {
        if (order_of(x, e) >= cut) atomicAdd(&sh->hist[bin_of(x)], by_weight ? share_of(x) : 1u);
      });
      cl.sync();
    }
    uint64_t above;
    const float width = inv_t / per_x;  // of a bin, in y
    const uint32_t bin = find_bin(false, want, &above, [&](int b, uint64_t sum) {
      return by_weight ? (uint64_t)((float)sum * expf(-width * b) * (float)(1 << (kFixed - 17))) : sum;
    });
    bool whole = false;
    if (!by_weight) {
      uint64_t held = 0;
      for (int r = 0; r < C; r++) held += bin < kBins ? *at(&sh->hist[bin], r) : 0;
      whole = above + held <= kList;
    }
    int got = -1;
    uint64_t before = above;
    if (bin < kBins) {
      uint64_t sum = 0;
      each([&](int e, float x) {
        const uint64_t o = order_of(x, e);
        if (o < cut) return;
        const int b = bin_of(x);
        if (b < (int)bin) {
          if (by_weight) sum += f_of(x);
          if (whole) put(o);
        } else if (b == (int)bin) {
          put(o);
        }
      });
      if (by_weight) before = cluster_sum(sum, 2);
      got = gather(!whole);
    }
    if (got >= 0 && whole) {
      *n = got;
      return cut;
    }
    if (got >= 0 && before < want) {
      // walk the gathered ones with exact sums
      constexpr int P = kList / kThreads;
      uint64_t v[P], mine = 0, all;
#pragma unroll
      for (int i = 0; i < P; i++) {
        const int k = tid * P + i;
        v[i] = k >= got ? 0 : by_weight ? f_of(of_key((uint32_t)(sh->list[k] >> 32))) : 1;
        mine += v[i];
      }
      uint64_t run = before + cta_scan(mine, sh, &all) - mine;
      if (before + all >= want) {
#pragma unroll
        for (int i = 0; i < P; i++) {
          if (run < want && want <= run + v[i]) sh->cut = sh->list[tid * P + i];
          run += v[i];
        }
        __syncthreads();
        return sh->cut;
      }
    }
    return select_slow(by_weight, want, cut);
  }

  // An element's weight as a share of its bin's upper one, in units of 2^-17.
  __device__ __forceinline__ uint32_t share_of(float x) const {
    const float d = x == top ? 0.f : (top - x) * per_x;
    const float z = (d - floorf(d)) * (inv_t / per_x);
    return d < (float)(kBins - 1) ? (uint32_t)((1.f - z + 0.5f * z * z) * 131072.f + 0.5f) : 131072u;
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
  return y - (float)log((double)total * (1.0 / (1ull << kFixed)));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char raw_smem[];
  Draw<T> d{{}, reinterpret_cast<Shared*>(raw_smem), cg::this_cluster()};
  Shared* sh = d.sh;
  const int C = d.C = (int)d.cl.num_blocks(), rank = d.rank = (int)d.cl.block_rank();
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

  float temp = a.temp_v ? a.temp_v[b] : a.temp;
  int k = a.top_k_v ? a.top_k_v[b] : a.top_k;
  const float top_p = a.top_p_v ? a.top_p_v[b] : a.top_p;
  const float min_p = fminf(a.min_p_v ? a.min_p_v[b] : a.min_p, 1.f);
  if (!(temp > 0.f)) {
    temp = 1.f;
    k = 1;
  }
  d.inv_t = 1.f / temp;
  // the bins reach 32 in y, past which nothing weighs anything, or 24 in x
  d.per_x = (float)kBins / fminf(32.f * temp, 24.f);
  const bool by_k = k > 0 && k < a.vocab, by_p = top_p < 1.f || top_p != top_p;

  // ---- the largest logit
  float top = -INFINITY;
  d.each([&](int, float x) { top = fmaxf(top, x); });
#pragma unroll
  for (int x = 16; x; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  if (lane == 0) sh->top[warp] = top;
  d.clear_hist();
  d.cl.sync();
  for (int i = lane; i < parts; i += 32) top = fmaxf(top, *d.at(&sh->top[i % kWarps], i / kWarps));
#pragma unroll
  for (int x = 16; x; x /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  d.top = top;
  if (top == -INFINITY) {  // nothing to draw from (the same for the whole cluster)
    if (rank == 0 && tid == 0) {
      a.token[b] = -1;
      a.logprob[b] = -INFINITY;
      a.kept[b] = 0;
    }
    d.cl.sync();
    return;
  }
  const float u = a.u[b];

  uint64_t cut = 0;  // kept are the tokens of at least this order
  int n = -1;
  if (by_k) cut = d.select(false, (uint64_t)k, 0, false, &n);
  if (n >= 0) {
    // ---- all that is left is in the list, in order: every CTA would find the same, the first one does
    if (rank == 0) {
      constexpr int P = kList / kThreads;
      const int m0 = k;
      uint64_t v[P], mine = 0, all;
      float w[P];
#pragma unroll
      for (int i = 0; i < P; i++) {
        const int j = tid * P + i;
        w[i] = j < m0 ? d.w_of(of_key((uint32_t)(sh->list[j] >> 32))) : 0.f;
        v[i] = fixed_of(w[i]);
        mine += v[i];
      }
      uint64_t run = cta_scan(mine, sh, &all) - mine;
      const uint64_t want = by_p ? goal_of(top_p, all) : UINT64_MAX;
      uint32_t c = 0;
#pragma unroll
      for (int i = 0; i < P; i++) {
        c += tid * P + i < m0 && run < want && w[i] >= min_p;
        run += v[i];
      }
      uint64_t kept;
      cta_scan(c, sh, &kept);
      // in index order now, each with its place in the list of logits
      const int m = (int)kept;
      for (int i = tid; i < m; i += kThreads)
        sh->mine[i] = (sh->list[i] & 0xffffffffull) << 32 | (uint32_t)i;
      __syncthreads();
      sort_list(sh->mine, m);
      mine = 0;
#pragma unroll
      for (int i = 0; i < P; i++) {
        const int j = tid * P + i;
        v[i] = j < m ? d.f_of(of_key((uint32_t)(sh->list[(uint32_t)sh->mine[j]] >> 32))) : 0;
        mine += v[i];
      }
      run = cta_scan(mine, sh, &all) - mine;
      const uint64_t aim = aim_of(u, all);
#pragma unroll
      for (int i = 0; i < P; i++) {
        if (run <= aim && aim < run + v[i]) {
          const uint64_t it = sh->mine[tid * P + i];
          a.token[b] = (int32_t)(0xffffffffu - (uint32_t)(it >> 32));
          a.logprob[b] = logprob_of(d.y_of(of_key((uint32_t)(sh->list[(uint32_t)it] >> 32))), all);
          a.kept[b] = (int32_t)kept;
        }
        run += v[i];
      }
    }
    d.cl.sync();  // no CTA leaves while another may read its shared memory
    return;
  }

  if (by_p) {
    // the weight of the first k, and the weight that min_p leaves of it
    if (by_k) {
      d.cl.sync();
      d.clear_hist();
    }
    const bool early = !(min_p > 0.f);  // with min_p the histogram is seldom needed
    uint64_t sum = 0, left = 0;
    d.each([&](int e, float x) {
      if (order_of(x, e) < cut) return;
      const float w = d.w_of(x);
      const uint64_t f = fixed_of(w);
      sum += f;
      if (early)
        atomicAdd(&sh->hist[d.bin_of(x)], d.share_of(x));
      else if (w >= min_p)
        left += f;
    });
    if (!early) {
      left = warp_sum(left);
      if (lane == 0) sh->warp_a[3][warp] = left;
    }
    sum = d.cluster_sum(sum, 0);
    const uint64_t want = goal_of(top_p, sum);
    bool binds = true;
    if (!early) {
      left = 0;
      for (int i = lane; i < parts; i += 32) left += *d.at(&sh->warp_a[3][i % kWarps], i / kWarps);
      binds = warp_sum(left) >= want;  // else min_p ends the prefix before
    }
    if (binds) cut = d.select(true, want, cut, early, &n);
  }

  // ---- the draw
  auto keeps = [&](int e, float x, uint64_t* f) {
    *f = 0;
    if (order_of(x, e) < cut) return false;
    const float w = d.w_of(x);
    if (w < min_p) return false;
    *f = fixed_of(w);
    return true;
  };
  uint64_t sum = 0;
  uint32_t c = 0;
  d.each([&](int e, float x) {
    uint64_t f;
    c += keeps(e, x, &f);
    sum += f;
  });
  sum = warp_sum(sum);
  c = (uint32_t)warp_sum(c);
  if (lane == 0) {
    sh->warp_a[1][warp] = sum;
    sh->warp_b[0][warp] = c;
  }
  d.cl.sync();
  // parts in index order: four to a lane
  constexpr int P = kMaxCluster * kWarps / 32;
  uint64_t v[P], mine = 0, kept = 0;
#pragma unroll
  for (int i = 0; i < P; i++) {
    const int j = lane * P + i;
    v[i] = j < parts ? *d.at(&sh->warp_a[1][j % kWarps], j / kWarps) : 0;
    kept += j < parts ? *d.at(&sh->warp_b[0][j % kWarps], j / kWarps) : 0;
    mine += v[i];
  }
  kept = warp_sum(kept);
  uint64_t incl = mine;
#pragma unroll
  for (int x = 1; x < 32; x *= 2) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, incl, x);
    if (lane >= x) incl += up;
  }
  const uint64_t total = __shfl_sync(0xffffffffu, incl, 31);
  const uint64_t aim = aim_of(u, total);
  uint64_t run = incl - mine, left = 0;
  bool ours = false;
#pragma unroll
  for (int i = 0; i < P; i++) {
    if (lane * P + i == part && run <= aim && aim < run + v[i]) {
      ours = true;
      left = aim - run;
    }
    run += v[i];
  }
  if (__any_sync(0xffffffffu, ours)) {
    // the first element of this warp's run whose running sum exceeds it
    left = warp_sum(left);
    for (int i0 = d.lo; i0 < d.hi; i0 += 32) {
      const int i = i0 + lane;
      float x[VEC];
      uint64_t f[VEC];
      mine = 0;
      if (i < d.hi) {
        d.row.load(i, x);
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          const int e = i * VEC - d.row.pad + j;
          f[j] = 0;
          if (e >= 0 && e < a.vocab) keeps(e, x[j], &f[j]);
          mine += f[j];
        }
      }
      incl = mine;
#pragma unroll
      for (int s = 1; s < 32; s *= 2) {
        const uint64_t up = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += up;
      }
      const uint64_t all = __shfl_sync(0xffffffffu, incl, 31);
      if (all <= left) {
        left -= all;
        continue;
      }
      if (incl > left && incl - mine <= left) {
        run = incl - mine;
        bool done = false;
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          run += f[j];
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
  d.cl.sync();  // no CTA leaves while another may read its shared memory
}

template <typename T>
cudaError_t launch(const Args& a, int lanes, cudaStream_t st) {
  // a row is split until a CTA has 4096 logits, or the CTAs fill the device;
  // a CTA's share stays below 2^17 logits (select_slow)
  int c = 1;
  while (c < kMaxCluster &&
         (a.vocab > (1 << 17) * c || (a.vocab > 4096 * c && (int64_t)lanes * c <= ops_sm_count())))
    c *= 2;
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
  static OpsOnce once;
  if (const int dev = ops_current(); !once(dev)) {
    const cudaError_t e =
        cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
    if (e != cudaSuccess) return e;
    once.set(dev);
  }
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a);
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
