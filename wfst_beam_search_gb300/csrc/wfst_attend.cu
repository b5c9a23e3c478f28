// wfst_attend.cu — attention of one new token per lane over a paged cache.
//
//   lane b sees n tokens of its cache: all `len` of them, or with a window w
//   the last w and the first `sinks` ones before them.  For each query head
//   S_j = scale * q . k_j,  o = sum_j softmax(S)_j v_j,  lse = log sum_j exp S_j
//   (a lane that sees nothing has o = 0, lse = -inf).  Query heads share the
//   key-value heads in equal runs.
//
// A pass has to read the visible keys and values once: 4 * D bytes per token
// and key-value head, for 4 * D flops per query head.  HBM bounds it.
//
// One pass over the keys with the running maximum and sum of the softmax.  The
// products run on matrix instructions, transposed: S^T = K Q^T takes 16 keys
// by 8 query heads, O^T = V^T P^T 16 elements of the value by 8 query heads,
// so that a run of up to 8 query heads wastes nothing of the keys' side and a
// key is read once for all of them.  P goes from the one's result to the
// other's operand through a transposing move, as its 16-bit rounding plus the
// rounding's rest: its error stays that of fp32.
//
// Work is split evenly whatever the lengths: a unit is 64 keys of one lane and
// head run, units are numbered through, and each CTA takes an equal range.  A
// CTA's warps each take 16 keys of a unit and copy them asynchronously into
// their own ring in shared memory, so they meet only where a lane's head ends.
// Where a head's units are shared among CTAs, each leaves its unscaled part in
// the workspace and the last one to arrive adds them up, in CTA order.
#include "wfst_ops.h"

namespace wfst {
namespace {

constexpr int kWarps = 4;
constexpr int kUnit = 16 * kWarps;  // keys of a unit
constexpr int kMaxGrid = 1024;      // CTAs the workspace has room for
constexpr int kColsMost = 16;       // query heads of a CTA's run at most
constexpr int kWidthMost = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// workspace: counters [kMaxGrid], then per CTA two parts of {m, l, o}
constexpr int64_t kPartFloats = 2 * kColsMost + kWidthMost * kColsMost;
constexpr int64_t kCounterBytes = kMaxGrid * 4;

struct Args {
  const void *q, *kc, *vc;
  const int32_t *table, *lens;
  void* o;
  float* lse;
  uint32_t* counters;
  float* parts;
  int64_t sq_b, sq_h, so_b, so_h, sl_b;
  int64_t ck_p, ck_s, ck_h, cv_p, cv_s, cv_h, st_b;
  int32_t lanes, hkv, share, runs, width, page, num_pages, window, sinks;
  uint32_t div_m;
  int32_t div_s;
  float scale2;  // scale * log2(e)
};

// What a lane sees: n tokens, the first `first` as they are, the others
// `shift` further on.
struct Seen {
  int n, first, shift, tiles;
};

__device__ __forceinline__ Seen seen(const Args& a, int b) {
  Seen s;
  const int64_t room = (int64_t)a.width * a.page;
  const int len = (int)max((int64_t)0, min((int64_t)a.lens[b], room));
  const int start = a.window > 0 ? max(0, len - a.window) : 0;
  s.first = min(a.sinks, start);
  s.shift = start - s.first;
  s.n = len - s.shift;
  s.tiles = max(1, (s.n + kUnit - 1) / kUnit);
  return s;
}

// Where a unit lies: lane, run of query heads, tile of the lane's keys.
struct Cursor {
  Seen s;
  int b, run, tile;
  __device__ __forceinline__ void next(const Args& a, int runs) {
    if (++tile < s.tiles) return;
    tile = 0;
    if (++run < runs) return;
    run = 0;
    if (++b < a.lanes) s = seen(a, b);
  }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 16 : 0;  // 0: sixteen zero bytes
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t turn8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2a(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

template <int D>
constexpr int kStages = D == 64 ? 6 : 3;
// rings, two warps' results at a segment's end, m and l of the warps
template <int D, int NT>
constexpr int kSmem = kWarps * kStages<D> * 2 * 16 * D * 2 + 2 * D * 8 * NT * 4 + kWarps * 2 * 8 * NT * 4;

// D: elements of a head; NT: runs of 8 * NT query heads.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32) attend_kernel(const Args a) {
  constexpr int S = kStages<D>, kTile = 16 * D * 2, kSlot = 2 * kTile, KS = D / 16, DT = D / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_scan[kWarps * 32 + 1];
  __shared__ int s_b, s_last;
  __shared__ int64_t s_base;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int runs = a.hkv * a.runs;

  // ---- this CTA's units: all lanes' tiles, numbered through
  const int per = (a.lanes + kWarps * 32 - 1) / (kWarps * 32);
  const int b_lo = min(a.lanes, tid * per), b_hi = min(a.lanes, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; b++) mine += seen(a, b).tiles;
  s_scan[tid + 1] = mine;
  if (tid == 0) s_scan[0] = 0;
  __syncthreads();
  if (warp == 0) {
    int64_t run_sum = 0;
    for (int i = 0; i < kWarps; i++) {
      int64_t v = s_scan[1 + i * 32 + lane];
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int64_t up = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += up;
      }
      v += run_sum;
      s_scan[1 + i * 32 + lane] = v;
      run_sum = __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  const int64_t units = s_scan[kWarps * 32] * runs;
  // CTAs that share the units; each of them has one at least
  const int64_t G = min((int64_t)gridDim.x, units);
  if (blockIdx.x >= G) return;
  const int64_t u0 = units * blockIdx.x / G, u1 = units * (blockIdx.x + 1) / G;
  {
    int64_t base = s_scan[tid] * runs;
    for (int b = b_lo; b < b_hi; b++) {
      const int64_t w = (int64_t)seen(a, b).tiles * runs;
      if (u0 >= base && u0 < base + w) s_b = b, s_base = base;
      base += w;
    }
  }
  __syncthreads();
  Cursor at;  // of the unit that is computed
  at.b = s_b;
  at.s = seen(a, at.b);
  int64_t seg0 = s_base;  // first unit of the current lane and run
  at.run = (int)((u0 - seg0) / at.s.tiles);
  seg0 += (int64_t)at.run * at.s.tiles;
  at.tile = (int)(u0 - seg0);

  // ---- the warp's ring
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (S * kSlot);
  float* xo = reinterpret_cast<float*>(smem + kWarps * S * kSlot);  // [2][NT][DT][32][4]
  float* xm = xo + 2 * D * 8 * NT;                                  // [warps][2][8 * NT]
  Cursor ahead = at;  // of the unit that is loaded next
  int id[2];
  int slot[2];
  const int row = g;  // a lane copies rows g and g + 8 of a tile, and masks the same ones
  auto look_up = [&]() {
#pragma unroll
    for (int r = 0; r < 2; r++) {
      const int i = ahead.tile * kUnit + warp * 16 + row + r * 8;
      id[r] = -1;
      slot[r] = 0;
      if (i < ahead.s.n) {
        const int key = i < ahead.s.first ? i : i + ahead.s.shift;
        const int pg = (int)(((uint64_t)(uint32_t)key * a.div_m) >> a.div_s);
        slot[r] = key - pg * a.page;
        id[r] = __ldg(a.table + ahead.b * a.st_b + pg);
      }
    }
  };
  uint32_t ok_bits = 0;  // two bits per slot of the ring
  int64_t u_ahead = u0;
  int put = 0;
  auto load_next = [&]() {
    if (u_ahead < u1) {
      const int h = ahead.run / a.runs;
      const uint32_t dst = ring + put * kSlot;
      uint32_t ok2 = 0;
#pragma unroll
      for (int r = 0; r < 2; r++) {
        const bool ok = (uint32_t)id[r] < (uint32_t)a.num_pages;
        ok2 |= ok ? 1u << r : 0u;
        const int64_t pg = ok ? id[r] : 0;
        const T* k = reinterpret_cast<const T*>(a.kc) + (ok ? pg * a.ck_p + slot[r] * a.ck_s + h * a.ck_h : 0);
        const T* v = reinterpret_cast<const T*>(a.vc) + (ok ? pg * a.cv_p + slot[r] * a.cv_s + h * a.cv_h : 0);
        const uint32_t line = dst + (row + r * 8) * (D * 2);
#pragma unroll
        for (int i = 0; i < D / 32; i++) {
          const int c = i * 4 + t;
          copy16(line + ((c ^ row) * 16), k + c * 8, ok);
        }
#pragma unroll
        for (int i = 0; i < D / 32; i++) {
          const int c = i * 4 + t;
          copy16(line + kTile + ((c ^ row) * 16), v + c * 8, ok);
        }
      }
      ok_bits = (ok_bits & ~(3u << (2 * put))) | ok2 << (2 * put);
      if (++u_ahead < u1) {
        ahead.next(a, runs);
        look_up();
      }
      put = put + 1 == S ? 0 : put + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  look_up();
#pragma unroll
  for (int i = 0; i < S - 1; i++) load_next();

  uint32_t qf[NT][KS][2];
  float o[NT][DT][4], m[NT][2], l[NT][2];
  auto begin_segment = [&]() {
    const int h = at.run / a.runs, c0 = (at.run % a.runs) * (8 * NT);
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const int c = c0 + n * 8 + g;
      const T* q = reinterpret_cast<const T*>(a.q) + at.b * a.sq_b + (int64_t)(h * a.share + c) * a.sq_h + 2 * t;
#pragma unroll
      for (int k = 0; k < KS; k++) {
        qf[n][k][0] = c < a.share ? __ldg(reinterpret_cast<const uint32_t*>(q + k * 16)) : 0u;
        qf[n][k][1] = c < a.share ? __ldg(reinterpret_cast<const uint32_t*>(q + k * 16 + 8)) : 0u;
      }
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; d++) o[n][d][0] = o[n][d][1] = o[n][d][2] = o[n][d][3] = 0.f;
    }
  };
  begin_segment();
  bool whole_start = at.tile == 0;
  bool from_u0 = true;  // the segment holds the range's first unit

  int get = 0;
  for (int64_t u = u0; u < u1; u++) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    __syncwarp();
    load_next();
    const uint32_t kt = ring + get * kSlot, vt = kt + kTile;
    const bool ok0 = ok_bits >> (2 * get) & 1u, ok1 = ok_bits >> (2 * get + 1) & 1u;
    get = get + 1 == S ? 0 : get + 1;

    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; n++) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    {
      const int r = (lane & 7) + (lane >> 3 & 1) * 8;
#pragma unroll
      for (int k = 0; k < KS; k++) {
        uint32_t f[4];
        ldm4(f, kt + r * (D * 2) + (((2 * k + (lane >> 4)) ^ (r & 7)) * 16));
#pragma unroll
        for (int n = 0; n < NT; n++) mma16816<T>(s[n], f[0], f[1], f[2], f[3], qf[n][k][0], qf[n][k][1]);
      }
    }
    uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
    for (int n = 0; n < NT; n++) {
      // heads 2t and 2t + 1 of keys g and g + 8
      s[n][0] = ok0 ? s[n][0] * a.scale2 : -INFINITY;
      s[n][1] = ok0 ? s[n][1] * a.scale2 : -INFINITY;
      s[n][2] = ok1 ? s[n][2] * a.scale2 : -INFINITY;
      s[n][3] = ok1 ? s[n][3] * a.scale2 : -INFINITY;
      float top[2] = {fmaxf(s[n][0], s[n][2]), fmaxf(s[n][1], s[n][3])};
      float keep[2];
#pragma unroll
      for (int c = 0; c < 2; c++) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], x));
        const float now = fmaxf(m[n][c], top[c]);
        const float ref = now == -INFINITY ? 0.f : now;
        keep[c] = exp2a(m[n][c] - ref);
        m[n][c] = now;
        top[c] = ref;
      }
      const float p0 = exp2a(s[n][0] - top[0]), p1 = exp2a(s[n][1] - top[1]);
      const float p2 = exp2a(s[n][2] - top[0]), p3 = exp2a(s[n][3] - top[1]);
      l[n][0] = l[n][0] * keep[0] + (p0 + p2);
      l[n][1] = l[n][1] * keep[1] + (p1 + p3);
      const uint32_t h0 = pack2<T>(p0, p1), h1 = pack2<T>(p2, p3);
      const float2 f0 = unpack2<T>(h0), f1 = unpack2<T>(h1);
      hi[n][0] = turn8x8(h0);
      hi[n][1] = turn8x8(h1);
      lo[n][0] = turn8x8(pack2<T>(p0 - f0.x, p1 - f0.y));
      lo[n][1] = turn8x8(pack2<T>(p2 - f1.x, p3 - f1.y));
#pragma unroll
      for (int d = 0; d < DT; d++) {
        o[n][d][0] *= keep[0];
        o[n][d][1] *= keep[1];
        o[n][d][2] *= keep[0];
        o[n][d][3] *= keep[1];
      }
    }
    {
      const int key = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
      for (int d = 0; d < DT; d++) {
        uint32_t f[4];
        ldm4t(f, vt + key * (D * 2) + (((2 * d + (lane >> 3 & 1)) ^ (key & 7)) * 16));
#pragma unroll
        for (int n = 0; n < NT; n++) {
          mma16816<T>(o[n][d], f[0], f[1], f[2], f[3], hi[n][0], hi[n][1]);
          mma16816<T>(o[n][d], f[0], f[1], f[2], f[3], lo[n][0], lo[n][1]);
        }
      }
    }

    const bool ends = at.tile + 1 == at.s.tiles;
    if (ends || u + 1 == u1) {
      // ---- the warps' parts become one, in warp 0
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int c = 0; c < 2; c++) {
#pragma unroll
          for (int x = 4; x < 32; x *= 2) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], x);
          if (g == 0) {
            xm[(warp * 2) * (8 * NT) + n * 8 + 2 * t + c] = m[n][c];
            xm[(warp * 2 + 1) * (8 * NT) + n * 8 + 2 * t + c] = l[n][c];
          }
        }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; n++) {
        float f[2];
#pragma unroll
        for (int c = 0; c < 2; c++) {
          const int col = n * 8 + 2 * t + c;
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; w++) top = fmaxf(top, xm[(w * 2) * (8 * NT) + col]);
          const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
          for (int w = 0; w < kWarps; w++)
            sum += xm[(w * 2 + 1) * (8 * NT) + col] * exp2a(xm[(w * 2) * (8 * NT) + col] - ref);
          f[c] = exp2a(m[n][c] - ref);
          m[n][c] = top;
          l[n][c] = sum;
        }
#pragma unroll
        for (int d = 0; d < DT; d++) {
          o[n][d][0] *= f[0];
          o[n][d][1] *= f[1];
          o[n][d][2] *= f[0];
          o[n][d][3] *= f[1];
        }
      }
#pragma unroll
      for (int half = 2; half >= 1; half /= 2) {
        if (warp >= half && warp < 2 * half) {
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int d = 0; d < DT; d++)
              reinterpret_cast<float4*>(xo)[(((warp - half) * NT + n) * DT + d) * 32 + lane] =
                  make_float4(o[n][d][0], o[n][d][1], o[n][d][2], o[n][d][3]);
        }
        __syncthreads();
        if (warp < half) {
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int d = 0; d < DT; d++) {
              const float4 v = reinterpret_cast<float4*>(xo)[((warp * NT + n) * DT + d) * 32 + lane];
              o[n][d][0] += v.x;
              o[n][d][1] += v.y;
              o[n][d][2] += v.z;
              o[n][d][3] += v.w;
            }
        }
        __syncthreads();
      }
      const bool whole = whole_start && ends;
      const int h = at.run / a.runs, c0 = (at.run % a.runs) * (8 * NT);
      bool write = whole;
      if (!whole) {
        // ---- this CTA's part goes to the workspace; the last one adds them up
        if (warp == 0) {
          float* part = a.parts + ((int64_t)blockIdx.x * 2 + (from_u0 ? 0 : 1)) * kPartFloats;
#pragma unroll
          for (int n = 0; n < NT; n++) {
            if (g == 0) {
#pragma unroll
              for (int c = 0; c < 2; c++) {
                part[n * 8 + 2 * t + c] = m[n][c];
                part[kColsMost + n * 8 + 2 * t + c] = l[n][c];
              }
            }
#pragma unroll
            for (int d = 0; d < DT; d++)
              reinterpret_cast<float4*>(part + 2 * kColsMost)[(n * DT + d) * 32 + lane] =
                  make_float4(o[n][d][0], o[n][d][1], o[n][d][2], o[n][d][3]);
          }
          __threadfence();
        }
        __syncthreads();
        // CTA c holds the units from units * c / G on: its number from a unit's
        const int64_t seg1 = seg0 + at.s.tiles;
        const int64_t c_first = ((seg0 + 1) * G - 1) / units, c_last = (seg1 * G - 1) / units;
        if (tid == 0) {
          const uint32_t n = (uint32_t)(c_last - c_first + 1);
          const uint32_t before = atomicAdd(a.counters + c_first, 1u);
          s_last = before + 1 == n;
          if (s_last) {
            a.counters[c_first] = 0;  // as the next call wants it
            __threadfence();
          }
        }
        __syncthreads();
        write = s_last != 0;
        if (write && warp == 0) {
#pragma unroll
          for (int n = 0; n < NT; n++) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int d = 0; d < DT; d++) o[n][d][0] = o[n][d][1] = o[n][d][2] = o[n][d][3] = 0.f;
          }
          for (int64_t c = c_first; c <= c_last; c++) {
            const int which = c > c_first || units * c / G == seg0 ? 0 : 1;
            const float* part = a.parts + (c * 2 + which) * kPartFloats;
#pragma unroll
            for (int n = 0; n < NT; n++) {
              float keep[2], add[2];
#pragma unroll
              for (int x = 0; x < 2; x++) {
                const float pm = __ldcg(part + n * 8 + 2 * t + x);
                const float pl = __ldcg(part + kColsMost + n * 8 + 2 * t + x);
                const float now = fmaxf(m[n][x], pm);
                const float ref = now == -INFINITY ? 0.f : now;
                keep[x] = exp2a(m[n][x] - ref);
                add[x] = exp2a(pm - ref);
                m[n][x] = now;
                l[n][x] = l[n][x] * keep[x] + pl * add[x];
              }
#pragma unroll
              for (int d = 0; d < DT; d++) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(part + 2 * kColsMost) + (n * DT + d) * 32 + lane);
                o[n][d][0] = o[n][d][0] * keep[0] + v.x * add[0];
                o[n][d][1] = o[n][d][1] * keep[1] + v.y * add[1];
                o[n][d][2] = o[n][d][2] * keep[0] + v.z * add[0];
                o[n][d][3] = o[n][d][3] * keep[1] + v.w * add[1];
              }
            }
          }
        }
      }
      if (write && warp == 0) {
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int x = 0; x < 2; x++) {
            const int c = c0 + n * 8 + 2 * t + x;
            if (c >= a.share) continue;
            const float inv = l[n][x] > 0.f || l[n][x] != l[n][x] ? 1.f / l[n][x] : 0.f;
            const int64_t head = (int64_t)h * a.share + c;
            T* out = reinterpret_cast<T*>(a.o) + at.b * a.so_b + head * a.so_h;
#pragma unroll
            for (int d = 0; d < DT; d++) {
              out[d * 16 + g] = from_f32<T>(o[n][d][x] * inv);
              out[d * 16 + g + 8] = from_f32<T>(o[n][d][x + 2] * inv);
            }
            if (a.lse && g == 0) a.lse[at.b * a.sl_b + head] = (m[n][x] + log2f(l[n][x])) * kLn2;
          }
      }
      if (u + 1 < u1) {
        seg0 += at.s.tiles;
        at.next(a, runs);
        begin_segment();
        whole_start = true;
        from_u0 = false;
      }
    } else {
      at.tile++;
    }
  }
}

template <typename T, int D, int NT>
cudaError_t launch(const Args& a, int64_t most_units, cudaStream_t st) {
  auto* fn = attend_kernel<T, D, NT>;
  constexpr int smem = kSmem<D, NT>;
  static OpsOnce once;
  static int resident = 1;  // CTAs of a multiprocessor
  if (const int dev = ops_current(); !once(dev)) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int v = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, fn, kWarps * 32, smem);
    if (e != cudaSuccess) return e;
    resident = v > 0 ? v : 1;
    once.set(dev);
  }
  int64_t grid = (int64_t)resident * ops_sm_count();
  if (grid > kMaxGrid) grid = kMaxGrid;
  if (grid > most_units) grid = most_units;
  fn<<<(int)grid, kWarps * 32, smem, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t by_share(Args& a, int64_t tiles, cudaStream_t st) {
  if (a.share <= 8) {
    a.runs = 1;
    return launch<T, D, 1>(a, tiles * a.hkv, st);
  }
  a.runs = (a.share + 15) / 16;
  return launch<T, D, 2>(a, tiles * a.hkv * a.runs, st);
}

template <typename T>
cudaError_t by_width(Args& a, int d, int64_t tiles, cudaStream_t st) {
  if (d == 64) return by_share<T, 64>(a, tiles, st);
  if (d == 128) return by_share<T, 128>(a, tiles, st);
  return by_share<T, 256>(a, tiles, st);
}

}  // namespace
}  // namespace wfst

using namespace wfst;

extern "C" int wfst_attend_size(int64_t* bytes) {
  if (!bytes) return api_fail(WFST_ERR_INVALID_ARG, "attend_size: NULL argument");
  *bytes = kCounterBytes + (int64_t)kMaxGrid * 2 * kPartFloats * 4;
  return WFST_OK;
}

extern "C" int wfst_attend_paged(const wfst_attend_args* r, void* stream) {
  if (!r) return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: NULL argument");
  if (r->dtype != WFST_F16 && r->dtype != WFST_BF16) return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: bad dtype");
  if (r->head_dim != 64 && r->head_dim != 128 && r->head_dim != 256)
    return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: head_dim must be 64, 128 or 256");
  if (r->lanes < 0 || r->q_heads < 0) return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: counts must be >= 0");
  if (r->kv_heads < 1 || r->q_heads % r->kv_heads)
    return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: q_heads must be a multiple of kv_heads");
  if (r->page_size < 1 || r->num_pages < 0 || r->table_width < 0)
    return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: page_size must be >= 1, num_pages and table_width >= 0");
  if ((int64_t)r->page_size * r->table_width > INT32_MAX - 1024)
    return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: page_size * table_width must stay below 2^31");
  if (r->window < 0 || r->sinks < 0) return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: window and sinks must be >= 0");
  if (!(r->scale == r->scale)) return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: scale must be a number");
  if (r->lanes == 0 || r->q_heads == 0) return WFST_OK;
  if (!r->q || !r->o || !r->lengths || !r->workspace || (r->table_width && !r->table) ||
      (r->num_pages && (!r->k_pages || !r->v_pages)))
    return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: NULL argument");
  for (const void* p : {r->q, r->k_pages, r->v_pages, (const void*)r->workspace})
    if (!aligned(p, 16)) return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: arrays must be 16-byte aligned");
  auto stride = [&](int64_t s, int64_t n) { return n > 1 ? s : 0; };
  Args a;
  a.sq_b = stride(r->q_stride[0], r->lanes), a.sq_h = stride(r->q_stride[1], r->q_heads);
  a.ck_p = stride(r->k_page_stride[0], r->num_pages), a.ck_s = stride(r->k_page_stride[1], r->page_size);
  a.cv_p = stride(r->v_page_stride[0], r->num_pages), a.cv_s = stride(r->v_page_stride[1], r->page_size);
  a.ck_h = stride(r->k_page_stride[2], r->kv_heads), a.cv_h = stride(r->v_page_stride[2], r->kv_heads);
  if ((a.sq_b | a.sq_h | a.ck_p | a.ck_s | a.ck_h | a.cv_p | a.cv_s | a.cv_h) & 7)
    return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: strides must be multiples of 8 elements");
  const int dev = ops_device(r->device, {r->q, r->k_pages, r->v_pages, r->table, r->lengths, r->o, r->lse, r->workspace});
  if (dev < 0) return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: every array must be device memory of one device");
  OpsDevice guard(dev);
  if (guard.err != cudaSuccess) return api_cuda_fail(guard.err, "attend_paged: device");
  a.q = r->q, a.kc = r->k_pages, a.vc = r->v_pages;
  a.table = r->table, a.lens = r->lengths;
  a.o = r->o, a.lse = r->lse;
  a.counters = reinterpret_cast<uint32_t*>(r->workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(r->workspace) + kCounterBytes);
  a.so_b = r->o_stride[0], a.so_h = r->o_stride[1], a.sl_b = r->lse_stride;
  a.st_b = stride(r->table_stride, r->lanes);
  a.lanes = r->lanes, a.hkv = r->kv_heads, a.share = r->q_heads / r->kv_heads, a.runs = 1;
  a.width = r->table_width, a.page = r->page_size, a.num_pages = r->num_pages;
  a.window = r->window, a.sinks = r->window ? r->sinks : 0;
  // key / page for key < 2^31: multiply by ceil(2^(31 + l) / page), l = ceil(log2 page)
  int l = 0;
  while ((int64_t)1 << l < r->page_size) l++;
  a.div_m = (uint32_t)((((uint64_t)1 << (31 + l)) + r->page_size - 1) / r->page_size);
  a.div_s = 31 + l;
  a.scale2 = r->scale * kLog2e;
  int64_t most = (int64_t)r->table_width * r->page_size;
  if (a.window && (int64_t)a.window + a.sinks < most) most = (int64_t)a.window + a.sinks;
  const int64_t tiles = (int64_t)a.lanes * (most / kUnit + 1);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = r->dtype == WFST_F16 ? by_width<__half>(a, r->head_dim, tiles, st)
                                             : by_width<__nv_bfloat16>(a, r->head_dim, tiles, st);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "attend_paged launch");
}
