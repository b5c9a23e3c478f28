// wfst_lowrank.cu — low-rank adapters of many requests beside a shared projection.
//
//   a = adapter[r],  t_j = scale[a] * sum_k x[r, k] * shrink[a, j, k]
//   out[r, n] = y[r, n] + sum_j t_j * expand[a, n, j]
//
// A pass has to read the adapters that some row uses, rank * (k + n) values each, and
// x and y, and write out: HBM bounds it, with few rows by the adapters, with many by x, y
// and out.
//
// A cluster of CTAs takes the rows of one adapter among 64 neighbouring rows: there
// are never more adapters than rows, a lane's rows lie side by side, and nothing has to be
// sorted.  Its CTAs share k for the first product and n for the second one; in between
// they exchange t through each other's shared memory, so that one launch does both.
// Which rows and adapter are its own a CTA finds by itself from the 64 numbers.
//
// Both products run on mma.sync, 16 rows at a time, with the adapters' values straight
// from memory (k is permuted within a step, alike on both sides, so that a lane loads 16
// or 8 bytes).  t is held in fp32 and goes into the second one in two 16-bit parts.  fp16
// has few exponents: there a row's t is multiplied by the power of two that brings
// its largest element to 2^14.
//
// What bounds it is the chain of one cluster: find the rows, first product, the warps' and
// the cluster's sums, second product, each some 2 to 5 us.  So what can be asked for early is
// (expand and y into the L2 cache during the first product, y before the second one), and
// two CTAs share a multiprocessor (with more registers for passes of 64 rows and one
// CTA, 4096 x 6144 x 4096 90 us instead of 50).  1 x 4096 x 4096 of rank 16 takes 6.5 us, 64 x
// 8192 x 8192 of 40 adapters of rank 64 27 (2.6 TB/s), 4096 x 6144 x 4096 of 16 of rank 16
// 50 (2.7 TB/s).
#include <cooperative_groups.h>

#include <type_traits>

#include "wfst_ops.h"

namespace cg = cooperative_groups;

namespace wfst {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRank = 128;
constexpr int kMaxCluster = 8;
constexpr int kTile = 64;   // neighbouring rows

struct Args {
  const void *y, *x, *shrink, *expand;
  const int32_t* adapter;
  const float* scales;
  void* out;
  int64_t sy, sx, so, ss_a, ss_j, se_a, se_n;
  int32_t rows, n, k, rank, adapters, ranks;  // ranks: rank up to a multiple of 16 (32, where it is more)
  int32_t same;  // out is y
};

// Shared memory, in floats, of a pass of P rows: sums of the warps; t, this CTA's part and
// all of it; t's parts, rows of 16-bit values with 8 more.
__host__ __device__ constexpr int red_floats(int P, int R, int ranks) { return 4 * P * (ranks < R ? ranks : R); }
__host__ __device__ constexpr int smem_floats(int P, int R, int ranks) {
  return red_floats(P, R, ranks) + 2 * P * ranks + P * (ranks + 8);
}

// Loads that nothing else is read with.
__device__ __forceinline__ uint4 load16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

// Eight neighbours of the 16 16-bit values of a and b, from the one at `first` (0 to 8) on.
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, uint32_t first) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (first & 8) return b;
#pragma unroll
  for (int i = 0; i < 6; i++) w[i] = first & 4 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; i++) w[i] = first & 2 ? w[i + 1] : w[i];
  const uint32_t by = first % 2 * 16;
  return make_uint4(__funnelshift_r(w[0], w[1], by), __funnelshift_r(w[1], w[2], by), __funnelshift_r(w[2], w[3], by),
                    __funnelshift_r(w[3], w[4], by));
}
// v of another lane, by all lanes of the warp.
__device__ __forceinline__ uint4 from_lane(const uint4& v, int lane) {
  return make_uint4(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane),
                    __shfl_sync(0xffffffffu, v.z, lane), __shfl_sync(0xffffffffu, v.w, lane));
}
// How many 16-bit values p is behind a 16-byte boundary.
__device__ __forceinline__ uint32_t behind(const uint16_t* p) { return (uint32_t)(reinterpret_cast<uintptr_t>(p) >> 1) & 7; }

// P rows to a pass; the first product has sums for R ranks at a time.  WIDE: y's and out's
// rows begin at 16 bytes.
template <typename T, int P, int R, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) lowrank_kernel(const Args a) {
  constexpr int MT = P / 16;
  extern __shared__ __align__(16) float smem[];
  __shared__ __align__(16) int ids[kTile], mine[kTile], none[kTile];
  __shared__ float lift[P];  // fp16: the powers of two to be taken off again
  __shared__ uint64_t s_leaders;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank_c = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  float* red = smem;
  float* part = red + red_floats(P, R, a.ranks);
  float* full = part + P * a.ranks;
  T* split = reinterpret_cast<T*>(full + P * a.ranks);  // [2][P][ranks + 8]
  const int row0 = blockIdx.z * kTile;
  ops_begin();
  ops_next();
  // ---- the tile's adapters, each at the first row that has it
  if (tid < kTile) {
    const int id = row0 + tid < a.rows ? ops_load(a.adapter + row0 + tid) : -1;
    ids[tid] = (uint32_t)id < (uint32_t)a.adapters ? id : -1;
    if (tid == 0) s_leaders = 0;
  }
  __syncthreads();
  if (tid < kTile) {
    const int id = ids[tid];
    const uint32_t alike = __match_any_sync(0xffffffffu, id);  // (by all lanes, whatever they have)
    bool first = id >= 0 && (alike & ((1u << lane) - 1)) == 0;
    for (int i = 0; i < warp * 32; i += 4) {  // nor among the warps before
      const int4 v = *reinterpret_cast<const int4*>(ids + i);
      if (v.x == id || v.y == id || v.z == id || v.w == id) first = false;
    }
    const uint32_t votes = __ballot_sync(0xffffffffu, first);
    if (lane == 0 && votes) atomicOr((unsigned long long*)&s_leaders, (unsigned long long)votes << (warp * 32));
  }
  __syncthreads();
  uint64_t leaders = s_leaders;
  auto share = [&](int blocks, int c) { return (int)((int64_t)blocks * c / C); };
  const int blocks_n = (a.n + 31) / 32, n_lo = share(blocks_n, rank_c), n_hi = share(blocks_n, rank_c + 1);
  // ---- rows without an adapter stay as they are: all clusters of the tile share them
  if (!a.same) {
    int count = 0;
    for (int h = 0; h < kTile / 32; h++) {
      const bool is_none = ids[h * 32 + lane] < 0 && row0 + h * 32 + lane < a.rows;
      const uint32_t is = __ballot_sync(0xffffffffu, is_none);
      if (warp == 0 && is_none) none[count + __popc(is & ((1u << lane) - 1))] = row0 + h * 32 + lane;
      count += __popc(is);
    }
    __syncthreads();
    // runs of eight values to a thread; where rows begin anywhere, of 256 to a warp, lane by lane
    const int each = WIDE ? (n_hi - n_lo) * 4 : (n_hi - n_lo + 7) / 8, end = min(n_hi * 32, a.n);
    const int by = WIDE ? 1 : 32, takes = kThreads / by;
    for (int i = blockIdx.y * takes + tid / by; i < count * each; i += gridDim.y * takes) {
      const int row = none[i / each], n = n_lo * 32 + i % each * (8 * by) + tid % by;
      const uint16_t* y = reinterpret_cast<const uint16_t*>(a.y) + row * a.sy + n;
      uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + row * a.so + n;
      if (WIDE && n + 8 <= a.n) {
        *reinterpret_cast<uint4*>(out) = load16(y);
      } else {
        uint16_t v[8];
#pragma unroll
        for (int z = 0; z < 8; z++) v[z] = n + z * by < end ? y[z * by] : 0;
#pragma unroll
        for (int z = 0; z < 8; z++)
          if (n + z * by < end) out[z * by] = v[z];
      }
    }
  }
  const int blocks_k = (a.k + 31) / 32, k_lo = share(blocks_k, rank_c), k_hi = share(blocks_k, rank_c + 1);

  // the tile's passes, of all its adapters, are dealt out to its clusters
  uint32_t until = blockIdx.y;  // passes until this cluster's next one
  for (; leaders; leaders &= leaders - 1) {
    const int id = ids[__ffsll((long long)leaders) - 1];
    int count = 0;
    uint32_t is[kTile / 32];
#pragma unroll
    for (int h = 0; h < kTile / 32; h++) {
      is[h] = __ballot_sync(0xffffffffu, ids[h * 32 + lane] == id);
      count += __popc(is[h]);
    }
    const uint32_t passes = (count + P - 1) / P, to_mine = until;
    while (until < passes) until += gridDim.y;
    until -= passes;
    if (to_mine >= passes) continue;
    // its rows
    __syncthreads();
    if (warp == 0) {
      int at = 0;
#pragma unroll
      for (int h = 0; h < kTile / 32; h++) {
        if (is[h] >> lane & 1) mine[at + __popc(is[h] & ((1u << lane) - 1))] = row0 + h * 32 + lane;
        at += __popc(is[h]);
      }
    }
    __syncthreads();
    const T* shrink = reinterpret_cast<const T*>(a.shrink) + id * a.ss_a;
    const T* expand = reinterpret_cast<const T*>(a.expand) + id * a.se_a;
    // the second product's values and y, on their way to the L2 cache meanwhile
    const int lines = ((min(n_hi * 32, a.n) - n_lo * 32) * (int)sizeof(T) + 127) / 128;
    auto fetch = [&]() {
      for (int n = n_lo * 32 + tid; n < min(n_hi * 32, a.n); n += kThreads)
        for (int j = 0; j < a.rank; j += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(expand + n * a.se_n + j));
      for (int i = warp; i < count; i += kWarps)
        for (int l = lane; l < lines; l += 32)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const T*>(a.y) + mine[i] * a.sy + n_lo * 32 +
                                                        l * (128 / (int)sizeof(T))));
    };
    const float scale = a.scales ? ops_load(a.scales + id) : 1.f;

    for (int p0 = (int)to_mine * P; p0 < count; p0 += (int)gridDim.y * P) {
      const int rows = min(P, count - p0);
      // ---- t, this CTA's share of k
      const T* xp[2 * MT];
#pragma unroll
      for (int m = 0; m < 2 * MT; m++) xp[m] = reinterpret_cast<const T*>(a.x) + mine[p0 + min(m * 8 + g, rows - 1)] * a.sx + t * 8;
      for (int r0 = 0; r0 < a.ranks; r0 += R) {
        const int nt = min(R, a.ranks - r0) / 8;  // runs of eight ranks
        float acc[MT][R / 8][4];
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
          for (int j = 0; j < R / 8; j++) acc[m][j][0] = acc[m][j][1] = acc[m][j][2] = acc[m][j][3] = 0.f;
        constexpr int B = R == 16 ? 2 : 1;  // blocks whose values are asked for at once, as many as registers hold
        for (int blk = k_lo + warp; blk < k_hi; blk += B * kWarps) {
          uint4 xv[B][2 * MT], sv[B][R / 8];
#pragma unroll
          for (int b = 0; b < B; b++) {
            const int k = (blk + b * kWarps) * 32;
            const bool in = blk + b * kWarps < k_hi && k + t * 8 < a.k;
#pragma unroll
            for (int m = 0; m < 2 * MT; m++) xv[b][m] = in && m * 8 < rows ? load16(xp[m] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < R / 8; j++)
              if (j < nt) {
                const int rank = r0 + j * 8 + g;
                sv[b][j] = in && rank < a.rank ? load16(shrink + rank * a.ss_j + k + t * 8) : make_uint4(0, 0, 0, 0);
              }
          }
          if (p0 == (int)to_mine * P && r0 == 0 && blk < k_lo + kWarps) fetch();
#pragma unroll
          for (int b = 0; b < B; b++)
#pragma unroll
            for (int j = 0; j < R / 8; j++)
              if (j < nt) {
#pragma unroll
                for (int m = 0; m < MT; m++) {
                  const uint4 lo = xv[b][2 * m], hi = xv[b][2 * m + 1];
                  mma16816<T>(acc[m][j], lo.x, hi.x, lo.y, hi.y, sv[b][j].x, sv[b][j].y);
                  mma16816<T>(acc[m][j], lo.z, hi.z, lo.w, hi.w, sv[b][j].z, sv[b][j].w);
                }
              }
        }
        // the warps' sums: four to four, then all of those, in order
        const int width = nt * 8;
        auto at = [&](int w, int m, int j, int half) { return red + ((w * P + m * 16 + half * 8 + g) * width + j * 8 + 2 * t); };
        __syncthreads();
        if (warp >= 4) {
#pragma unroll
          for (int m = 0; m < MT; m++)
#pragma unroll
            for (int j = 0; j < R / 8; j++)
              if (j < nt) {
                *reinterpret_cast<float2*>(at(warp - 4, m, j, 0)) = make_float2(acc[m][j][0], acc[m][j][1]);
                *reinterpret_cast<float2*>(at(warp - 4, m, j, 1)) = make_float2(acc[m][j][2], acc[m][j][3]);
              }
        }
        __syncthreads();
        if (warp < 4) {
#pragma unroll
          for (int m = 0; m < MT; m++)
#pragma unroll
            for (int j = 0; j < R / 8; j++)
              if (j < nt)
#pragma unroll
                for (int half = 0; half < 2; half++) {
                  float2* p = reinterpret_cast<float2*>(at(warp, m, j, half));
                  const float2 v = *p;
                  *p = make_float2(v.x + acc[m][j][2 * half], v.y + acc[m][j][2 * half + 1]);
                }
        }
        __syncthreads();
        for (int i = tid; i < P * width; i += kThreads) {
          const int r = i / width, j = i % width;
          part[r * a.ranks + r0 + j] = (red[i] + red[P * width + i]) + (red[2 * P * width + i] + red[3 * P * width + i]);
        }
      }
      // ---- the cluster's: each CTA adds up its share of t, in order, and gives it to all
      if (C > 1) {
        cl.sync();
        const float* from[kMaxCluster];
        float* to[kMaxCluster];
#pragma unroll
        for (int c = 0; c < kMaxCluster; c++) {
          from[c] = cl.map_shared_rank(part, c < C ? c : 0);
          to[c] = cl.map_shared_rank(full, c < C ? c : 0);
        }
        for (int i = rank_c * kThreads + tid; i < rows * a.ranks; i += C * kThreads) {
          float v[kMaxCluster];
#pragma unroll
          for (int c = 0; c < kMaxCluster; c++) v[c] = c < C ? from[c][i] : 0.f;
          float sum = v[0];
#pragma unroll
          for (int c = 1; c < kMaxCluster; c++) sum += v[c];
          sum *= scale;
#pragma unroll
          for (int c = 0; c < kMaxCluster; c++)
            if (c < C) to[c][i] = sum;
        }
        cl.sync();
      } else {
        __syncthreads();
        for (int i = tid; i < rows * a.ranks; i += kThreads) full[i] = part[i] * scale;
        __syncthreads();
      }
      // ---- in two parts; a warp takes a row at a time
      for (int r = warp; r < P; r += kWarps) {
        float up = 1.f;
        if (std::is_same_v<T, __half>) {
          float top = 0.f;
          if (r < rows)
            for (int j = lane; j < a.ranks; j += 32) top = fmaxf(top, fabsf(full[r * a.ranks + j]));
          const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
          // 2^14 / 2^exponent, and its inverse, both within fp32's exponents
          const int e = min(max((int)(most >> 23) - 127, -112), 126);
          if (most && most < 0x7f800000u) up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
          if (lane == 0) lift[r] = most && most < 0x7f800000u ? __uint_as_float((uint32_t)(127 - 14 + e) << 23) : 1.f;
        }
        for (int j = lane; j < a.ranks; j += 32) {
          const float v = r < rows ? full[r * a.ranks + j] * up : 0.f;
          const T hi = from_f32<T>(v);
          split[r * (a.ranks + 8) + j] = hi;
          split[(P + r) * (a.ranks + 8) + j] = from_f32<T>(v - to_f32(hi));
        }
      }
      __syncthreads();
      // ---- y plus t times expand: 32 outputs to a warp at a time, of which a lane has eight
      // neighbours in the end (run q of eight holds outputs 8 i + 2 q and 8 i + 2 q + 1)
      // steps of S ranks, of which a lane has S / 4 neighbours on either side; U of them are asked for at once
      constexpr int S = R == 16 ? 16 : 32, U = R / S;
      using Run = std::conditional_t<S == 16, uint2, uint4>;
      // Rows that do not begin at 16 bytes: of a block inside the row, four neighbouring lanes load the
      // aligned pieces that hold a row's values, and shift them.  A fifth piece is needed for the last
      // values: lane t has that of its rows' t-th.  (What else is in the outer pieces, which another warp
      // may be writing where out is y, is not used.)  640 x 7517 x 864 of rank 16 takes 27 us so, 47 with
      // each value loaded and stored by itself; with 7520 it takes 16.
      struct Block {
        uint4 y[MT][2], more;
        Run e[U][4];
      };
      // up to eight rows: the upper eight of the product's 16 are the same rows' second parts
      const bool beside = P == 16 && rows <= 8;
      auto wide = [&](int n) { return WIDE && n + 8 <= a.n; };
      auto ask_e = [&](Block& v, int n0, int s0) {
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const T* ep = expand + (int64_t)min(n0 + g / 2 * 8 + 2 * q + g % 2, a.n - 1) * a.se_n + s0 + t * (S / 4);
#pragma unroll
          for (int u = 0; u < U; u++)
            v.e[u][q] = s0 + u * S + t * (S / 4) < a.rank ? *reinterpret_cast<const Run*>(ep + u * S) : Run{};
        }
      };
      auto inside = [&](int n0) { return !WIDE && n0 >= 8 && n0 + 40 <= a.n; };
      auto ask = [&](Block& v, int blk) {
        const int n0 = blk * 32, n = n0 + t * 8;
        if (inside(n0)) {
          v.more = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int m = 0; m < MT; m++)
#pragma unroll
            for (int half = 0; half < 2; half++) {
              const int r = m * 16 + half * 8 + g;
              v.y[m][half] = make_uint4(0, 0, 0, 0);
              if (r >= rows) continue;  // (of that lane)
              const uint16_t* y = reinterpret_cast<const uint16_t*>(a.y) + mine[p0 + r] * a.sy + n0;
              const uint32_t d = behind(y);
              v.y[m][half] = load16(y - d + t * 8);
              if (t == 2 * m + half && d) v.more = load16(y - d + 32);
            }
          ask_e(v, n0, 0);
          return;
        }
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
          for (int half = 0; half < 2; half++) {
            const int r = m * 16 + half * 8 + g;
            v.y[m][half] = make_uint4(0, 0, 0, 0);
            if (r >= rows || n >= a.n) continue;
            const uint16_t* y = reinterpret_cast<const uint16_t*>(a.y) + mine[p0 + r] * a.sy + n;
            if (wide(n)) {
              v.y[m][half] = load16(y);
            } else {
              uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
              for (int z = 0; z < 8; z++)
                if (n + z < a.n) w[z / 2] |= (uint32_t)y[z] << z % 2 * 16;
              v.y[m][half] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        ask_e(v, n0, 0);
      };
      auto finish = [&](Block& v, int blk) {
        const int n0 = blk * 32, n = n0 + t * 8;
        float acc[MT][4][4];
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
          for (int q = 0; q < 4; q++) acc[m][q][0] = acc[m][q][1] = acc[m][q][2] = acc[m][q][3] = 0.f;
        for (int s0 = 0; s0 < a.ranks; s0 += S * U) {
          if (s0) ask_e(v, n0, s0);
#pragma unroll
          for (int u = 0; u < U; u++) {
            const int s = s0 + u * S;
            if (s >= a.ranks) break;
            auto multiply = [&](int m, const Run& lo, const Run& hi) {
#pragma unroll
              for (int q = 0; q < 4; q++) {
                mma16816<T>(acc[m][q], lo.x, hi.x, lo.y, hi.y, v.e[u][q].x, v.e[u][q].y);
                if constexpr (S == 32) mma16816<T>(acc[m][q], lo.z, hi.z, lo.w, hi.w, v.e[u][q].z, v.e[u][q].w);
              }
            };
            auto row = [&](int r) { return *reinterpret_cast<const Run*>(split + r * (a.ranks + 8) + s + t * (S / 4)); };
            if (beside) {
              multiply(0, row(g), row(P + g));
              continue;
            }
#pragma unroll
            for (int m = 0; m < MT; m++) {
              if (m * 16 >= rows) break;
#pragma unroll
              for (int h = 0; h < 2; h++) multiply(m, row(h * P + m * 16 + g), row(h * P + m * 16 + 8 + g));
            }
          }
        }
        if (beside) {
#pragma unroll
          for (int q = 0; q < 4; q++) acc[0][q][0] += acc[0][q][2], acc[0][q][1] += acc[0][q][3];
        }
        if (inside(n0)) {  // (all lanes take part in the exchange)
#pragma unroll
          for (int m = 0; m < MT; m++)
#pragma unroll
            for (int half = 0; half < 2; half++) {
              if (m * 16 + half * 8 >= rows) break;  // (of all lanes)
              const int r = m * 16 + half * 8 + g, row = mine[p0 + min(r, rows - 1)];
              const uint4 next = from_lane(v.y[m][half], lane + 1), last = from_lane(v.more, lane - t + 2 * m + half);
              const uint4 w = shifted(v.y[m][half], t < 3 ? next : last,
                                      behind(reinterpret_cast<const uint16_t*>(a.y) + row * a.sy + n0));
              const float down = std::is_same_v<T, __half> && r < rows ? lift[r] : 1.f;
              const uint32_t u[4] = {w.x, w.y, w.z, w.w};
              uint32_t o[4];
#pragma unroll
              for (int q = 0; q < 4; q++) {
                const float2 f = unpack2<T>(u[q]);
                o[q] = pack2<T>(f.x + acc[m][q][2 * half] * down, f.y + acc[m][q][2 * half + 1] * down);
              }
              // a lane stores the piece that its first values are in, from the boundary on; the first one's,
              // and what lies behind the last boundary, is one piece too, whose ends the outer lanes store
              const uint4 own = make_uint4(o[0], o[1], o[2], o[3]), before = from_lane(own, lane ^ t ^ ((t + 3) & 3));
              uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + row * a.so + n0;
              const uint32_t d = behind(out);
              const uint4 piece = shifted(before, own, 8 - d), ends = from_lane(piece, lane - t);
              if (r >= rows) continue;
              out += t * 8 - (int)d;
              if (t > 0 || d == 0) *reinterpret_cast<uint4*>(out) = piece;
              if (d && (t == 0 || t == 3)) {
                const bool head = t == 0;
                const uint32_t few = head ? 8 - d : d;
                if (!head) out += 8;
                if (few & 4) *reinterpret_cast<uint2*>(out + (head ? 4 : 0)) = head ? make_uint2(ends.z, ends.w) : make_uint2(ends.x, ends.y);
                if (few & 2) {
                  const uint32_t low = head ? ends.y : ends.x, high = head ? ends.w : ends.z;
                  *reinterpret_cast<uint32_t*>(out + (d & 4) + (head ? 2 : 0)) = d & 4 ? high : low;
                }
                if (few & 1) {
                  const uint32_t odd = d & 4 ? (d & 2 ? ends.w : ends.z) : d & 2 ? ends.y : ends.x;
                  out[head ? d : d - 1] = (uint16_t)(head ? odd >> 16 : odd);
                }
              }
            }
          return;
        }
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
          for (int half = 0; half < 2; half++) {
            const int r = m * 16 + half * 8 + g;
            if (r >= rows || n >= a.n) continue;
            const float down = std::is_same_v<T, __half> ? lift[r] : 1.f;
            const uint32_t w[4] = {v.y[m][half].x, v.y[m][half].y, v.y[m][half].z, v.y[m][half].w};
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; q++) {
              const float2 f = unpack2<T>(w[q]);
              o[q] = pack2<T>(f.x + acc[m][q][2 * half] * down, f.y + acc[m][q][2 * half + 1] * down);
            }
            uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + mine[p0 + r] * a.so + n;
            if (wide(n)) {
              *reinterpret_cast<uint4*>(out) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
#pragma unroll
              for (int z = 0; z < 8; z++)
                if (n + z < a.n) out[z] = (uint16_t)(o[z / 2] >> z % 2 * 16);
            }
          }
      };
#pragma unroll 1
      for (int blk = n_lo + warp; blk < n_hi; blk += kWarps) {
        Block v;
        ask(v, blk);  // (y among it: it takes the longest, and out may be y)
        finish(v, blk);
      }
      __syncthreads();  // t's parts have been read
    }
  }
  if (C > 1) cl.sync();  // no CTA leaves while another may read its shared memory
}

template <typename T, int P, int R, bool WIDE>
cudaError_t launch(const Args& a, cudaStream_t st) {
  auto* fn = lowrank_kernel<T, P, R, WIDE>;
  constexpr int most = smem_floats(P, R, R == 16 ? 16 : kMaxRank) * 4;
  static OpsOnce once;
  if (const int dev = ops_current(); !once(dev)) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    once.set(dev);
  }
  // A CTA has 256 of k or n at least.  A tile's adapters are shared among clusters while
  // there are places for them.
  int C = 1;
  while (C < kMaxCluster && C * 512 <= (a.k > a.n ? a.k : a.n)) C *= 2;
  const int tiles = (a.rows + kTile - 1) / kTile;
  const int most_rows = a.rows < kTile ? a.rows : kTile;
  int among = a.adapters > (most_rows + P - 1) / P ? a.adapters : (most_rows + P - 1) / P;  // passes of a tile, or hardly more
  if (among > most_rows) among = most_rows;
  const int64_t room = 4ll * ops_sm_count() / ((int64_t)tiles * C);
  if (among > room && tiles > 1) among = room > 1 ? (int)room : 1;
  return ops_launch(fn, dim3(C, among, tiles), kThreads, smem_floats(P, R, a.ranks) * 4, C, st, a);
}

// Rows to a pass: 16 where an adapter will hardly have more of a tile's, as in a batch of
// one token per lane; otherwise 32 (4096 x 6144 x 4096 50 us, with 16 76).
template <typename T, bool WIDE>
cudaError_t by_rows(const Args& a, cudaStream_t st) {
  const bool few = a.rows <= 16 || a.rows <= (int64_t)a.adapters * 12;
  if (a.ranks == 16) return few ? launch<T, 16, 16, WIDE>(a, st) : launch<T, 32, 16, WIDE>(a, st);
  return few ? launch<T, 16, 64, WIDE>(a, st) : launch<T, 32, 32, WIDE>(a, st);
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
  if (r->rows > 65535 * kTile) return api_fail(WFST_ERR_INVALID_ARG, "add_lowrank: too many rows");
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
  a.ranks = a.rank <= 16 ? 16 : (a.rank + 31) / 32 * 32;
  a.same = a.out == a.y && a.so == a.sy;
  const bool wide = aligned(a.y, 16) && aligned(a.out, 16) && a.sy % 8 == 0 && a.so % 8 == 0;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = r->dtype == WFST_F16 ? (wide ? by_rows<__half, true>(a, st) : by_rows<__half, false>(a, st))
                                             : (wide ? by_rows<__nv_bfloat16, true>(a, st) : by_rows<__nv_bfloat16, false>(a, st));
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "add_lowrank launch");
}
