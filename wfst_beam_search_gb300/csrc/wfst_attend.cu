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
// other's operand through a transposing move, in 16-bit parts that add up to its
// fp32 value: two of fp16, three of bf16.  (With two of bf16, 2^-18 of P is lost;
// the third costs 0 to 0.5% with up to 8 query heads to a key-value head and 4 to 6%
// with 12: 32 lanes of 4096 tokens with heads of 256 216 to 228 us.)
//
// Work is split evenly whatever the lengths: a unit is 16 keys for each of a
// CTA's warps, of one lane and head run; units are numbered through, and each CTA
// takes an equal range.  A warp copies its keys and values asynchronously into a
// ring of its own in shared memory, so warps meet only where a lane's head ends.
// Where a head's units are shared among CTAs, each leaves its unscaled part in
// the workspace and the last one to arrive adds them up, in CTA order.
//
// Heads of 128, 32 or 64 query and 8 key-value heads: 2 lanes of 100000 to 131072
// tokens (0.95 to 0.97 GB) take 153 to 160 us, 6.2 TB/s, 64 lanes of 1 to 8192 (1.0
// to 1.08 GB) 174 to 179, 128 lanes with a window of 2047 (1.07 GB) 173 to 178: 83
// to 94% of a plain copy's rate.  One lane of 500 tokens takes 7.5 us: finding the units,
// two round trips to memory (page, keys), the join.
//
// wfst_prefix.cu has this kernel leave m, l and o unscaled (PRE), for lanes that follow a
// shared prefix.
#include "wfst_ops.h"

namespace wfst {
namespace {

constexpr int kLeastUnit = 64;      // keys of a unit, at least
constexpr int kMaxGrid = 1024;      // CTAs the workspace has room for
constexpr int kColsMost = 16;       // query heads of a CTA's run at most
constexpr int kWidthMost = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// P's parts are its rounding to T, the rest's, and bf16's second rest's.  fp16 has
// no exponents below 2^-24, at which a weight 17 below the largest score would be
// lost: there P, and with it l and o, is held times 2^15, so that the largest is
// 2^15 and what is lost below 2^-40 of it.
template <typename T>
constexpr float kLift = std::is_same_v<T, __half> ? 15.f : 0.f;

// workspace: counters [kMaxGrid], then per CTA two parts of {m, l, o}
constexpr int64_t kPartFloats = 2 * kColsMost + kWidthMost * kColsMost;
constexpr int64_t kCounterBytes = kMaxGrid * 4;
static_assert(kCounterBytes == WFST_ATTEND_ZEROED, "the parts are written before they are read");

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
  int32_t o_even;  // o's pairs of elements are 4-byte aligned
  float* own;  // PRE: m [own_rows], l [own_rows], o [own_rows][D]; rows by key-value head, lane, head
  int64_t own_rows;
};

// What a lane sees: n tokens, the first `first` as they are, the others
// `shift` further on.
struct Seen {
  int n, first, shift, tiles;
};

template <int UNIT>
__device__ __forceinline__ Seen seen(const Args& a, int b) {
  Seen s;
  const int64_t room = (int64_t)a.width * a.page;
  const int len = (int)max((int64_t)0, min((int64_t)a.lens[b], room));
  const int start = a.window > 0 ? max(0, len - a.window) : 0;
  s.first = min(a.sinks, start);
  s.shift = start - s.first;
  s.n = len - s.shift;
  s.tiles = max(1, (s.n + UNIT - 1) / UNIT);
  return s;
}

// Where a unit lies: lane, run of query heads, tile of the lane's keys.
template <int UNIT>
struct Cursor {
  Seen s;
  int b, run, tile;
  __device__ __forceinline__ void next(const Args& a, int runs) {
    if (++tile < s.tiles) return;
    tile = 0;
    if (++run < runs) return;
    run = 0;
    if (++b < a.lanes) s = seen<UNIT>(a, b);
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

// Warps of a CTA, and 16-row tiles in a warp's ring, of which keys and values
// take one each: what 227 KB hold for heads of 256, and what lets two CTAs (three
// for heads of 64) share a multiprocessor otherwise.  With a tile less each, 74
// lanes of 450 tokens with heads of 256 take 47 instead of 43 us, 2 x 131072 160
// instead of 158; with eight warps for heads of 128, 64 lanes of 1 to 8192 tokens
// take 190 instead of 177 (2 x 131072 154 instead of 158).
template <int D>
constexpr int kWarps = D == 256 ? 8 : 4;
template <int D>
constexpr int kRing = D == 64 ? 8 : D == 128 ? 5 : 3;
// rings, two warps' results at a segment's end, m and l of the warps
template <int D, int NT>
constexpr int kSmem = kWarps<D> * kRing<D> * 16 * D * 2 + 2 * D * 8 * NT * 4 + kWarps<D> * 2 * 8 * NT * 4;

// D: elements of a head; NT: runs of 8 * NT query heads.  PRE: m, l and o are left
// unscaled for wfst_prefix.cu, whose kernel before this one may still run: this one
// ends after it.
template <typename T, int D, int NT, bool PRE>
__global__ void __launch_bounds__(kWarps<D> * 32) attend_kernel(const Args a) {
  constexpr int W = kWarps<D>, UNIT = 16 * W, S = kRing<D>, kTile = 16 * D * 2, KS = D / 16, DT = D / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint32_t s_last[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int runs = a.hkv * a.runs;
  // (with PRE the kernel before has waited itself for what this one reads)
  if (!PRE) ops_begin();
  ops_next();

  // ---- this CTA's units: all lanes' tiles, numbered through (each warp for itself)
  uint32_t units = 0;
#pragma unroll 4
  for (int b = lane; b < a.lanes; b += 32) units += seen<UNIT>(a, b).tiles;
  units = __reduce_add_sync(0xffffffffu, units) * runs;
  // CTAs that share the units; each of them has one at least
  const uint32_t G = min(gridDim.x, units), each = units / G, more = units - each * G;
  if (blockIdx.x >= G) {
    if (PRE) ops_begin();
    return;
  }
  auto first_of = [&](uint32_t c) { return c * each + min(c, more); };
  auto cta_of = [&](uint32_t u) {
    const uint32_t at = more * (each + 1);
    return u < at ? u / (each + 1) : more + (u - at) / each;
  };
  const uint32_t u0 = first_of(blockIdx.x), u1 = first_of(blockIdx.x + 1);
  Cursor<UNIT> at;  // of the unit that is computed
  uint32_t seg0 = 0;  // first unit of the current lane and run
  for (int b0 = 0;; b0 += 32) {
    const uint32_t mine = b0 + lane < a.lanes ? seen<UNIT>(a, b0 + lane).tiles * runs : 0;
    uint32_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, seg0 + incl > u0);
    if (past) {
      at.b = b0 + __ffs(past) - 1;
      seg0 += __shfl_sync(0xffffffffu, incl - mine, __ffs(past) - 1);
      break;
    }
    seg0 += __shfl_sync(0xffffffffu, incl, 31);
  }
  at.s = seen<UNIT>(a, at.b);
  at.run = (u0 - seg0) / at.s.tiles;
  seg0 += at.run * at.s.tiles;
  at.tile = u0 - seg0;

  // ---- the warp's ring
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (S * kTile);
  float* xo = reinterpret_cast<float*>(smem + W * S * kTile);  // [2][NT][DT][32][4]
  float* xm = xo + 2 * D * 8 * NT;                                  // [warps][2][8 * NT]
  Cursor<UNIT> ahead = at;  // of the unit that is looked up last
  struct Rows {  // of the pool, that a lane copies: rows g and g + 8 of a tile, which it also masks
    int id[2], slot[2], head;
  };
  auto look_up = [&]() {
    Rows r;
    r.head = ahead.run / a.runs;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int j = ahead.tile * UNIT + warp * 16 + g + i * 8;
      r.id[i] = -1;
      r.slot[i] = 0;
      if (j < ahead.s.n) {
        const int key = j < ahead.s.first ? j : j + ahead.s.shift;
        const int pg = (int)(((uint64_t)(uint32_t)key * a.div_m) >> a.div_s);
        r.slot[i] = key - pg * a.page;
        r.id[i] = ops_load(a.table + ahead.b * a.st_b + pg);
      }
    }
    return r;
  };
  uint32_t ok_bits = 0;  // two bits per unit in flight
  int put = 0;
  auto copy_tile = [&](const Rows& r, const void* pool, int64_t s_p, int64_t s_s, int64_t s_h) {
    const uint32_t dst = ring + put * kTile + g * (D * 2);
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const bool ok = (uint32_t)r.id[i] < (uint32_t)a.num_pages;
      const T* from = reinterpret_cast<const T*>(pool) + (ok ? r.id[i] * s_p + r.slot[i] * s_s + r.head * s_h : 0);
#pragma unroll
      for (int j = 0; j < D / 32; j++) copy16(dst + i * (16 * D) + (((j * 4 + t) ^ g) * 16), from + (j * 4 + t) * 8, ok);
    }
    put = put + 1 == S ? 0 : put + 1;
  };
  auto copy_keys = [&](const Rows& r, uint32_t u) {
    copy_tile(r, a.kc, a.ck_p, a.ck_s, a.ck_h);
    const uint32_t ok2 = ((uint32_t)r.id[0] < (uint32_t)a.num_pages ? 1u : 0u) | ((uint32_t)r.id[1] < (uint32_t)a.num_pages ? 2u : 0u);
    ok_bits = (ok_bits & ~(3u << (2 * (u & 7)))) | ok2 << (2 * (u & 7));
  };
  auto copy_values = [&](const Rows& r) { copy_tile(r, a.vc, a.cv_p, a.cv_s, a.cv_h); };
  // the first S - 1 tiles: all their page numbers at once, then the copies
  constexpr int F = S / 2;  // units they belong to
  Rows rows[F + 1] = {};
#pragma unroll
  for (int i = 0; i <= F; i++)
    if (u0 + i < u1) {
      if (i) ahead.next(a, runs);
      rows[i] = look_up();
    }
#pragma unroll
  for (int i = 0; i < S - 1; i++) {
    if (u0 + i / 2 < u1) {
      if (i % 2)
        copy_values(rows[i / 2]);
      else
        copy_keys(rows[i / 2], i / 2);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // after that tile by tile, while the next unit's page numbers are on their way
  Rows now = rows[S % 2 ? F : F - 1], next = rows[F];
  uint32_t u_ahead = u0 + (S % 2 ? F : F - 1);
  auto copy_next = [&](bool values) {
    if (u_ahead < u1) {
      if (values) {
        copy_values(now);
        now = next;
        u_ahead++;
      } else {
        copy_keys(now, u_ahead - u0);
        if (u_ahead + 1 < u1) {
          ahead.next(a, runs);
          next = look_up();
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  uint32_t qf[NT][KS][2];
  float o[NT][DT][4], m[NT][2], l[NT][2];
  // the next segment's queries, on their way to L1 while this one's keys are read
  auto fetch_queries = [&]() {
    int b = at.b, run = at.run + 1;
    if (run == runs) run = 0, b++;
    if (b >= a.lanes) return;
    const int h = run / a.runs, c0 = (run % a.runs) * (8 * NT);
    for (int i = lane; i < 8 * NT * (D / 64); i += 32) {
      const int c = c0 + i / (D / 64);
      if (c >= a.share) continue;
      const T* q = reinterpret_cast<const T*>(a.q) + b * a.sq_b + (int64_t)(h * a.share + c) * a.sq_h + i % (D / 64) * 64;
      asm volatile("prefetch.global.L1 [%0];" ::"l"(q));
    }
  };
  auto begin_segment = [&]() {
    const int h = at.run / a.runs, c0 = (at.run % a.runs) * (8 * NT);
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const int c = c0 + n * 8 + g;
      const T* q = reinterpret_cast<const T*>(a.q) + at.b * a.sq_b + (int64_t)(h * a.share + c) * a.sq_h + 2 * t;
#pragma unroll
      for (int k = 0; k < KS; k++) {
        qf[n][k][0] = c < a.share ? ops_load(reinterpret_cast<const uint32_t*>(q + k * 16)) : 0u;
        qf[n][k][1] = c < a.share ? ops_load(reinterpret_cast<const uint32_t*>(q + k * 16 + 8)) : 0u;
      }
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; d++) o[n][d][0] = o[n][d][1] = o[n][d][2] = o[n][d][3] = 0.f;
    }
    if (warp == 0) fetch_queries();
  };
  begin_segment();
  // 16 elements from 16 * d on of the eight heads of run n: rows g and g + 8,
  // columns 2t and 2t + 1 of the transposed result
  auto put_out = [&](int b, int run, int n, int d, const float (&w)[4], const float (&wl)[2]) {
    const float i0 = wl[0] > 0.f || wl[0] != wl[0] ? 1.f / wl[0] : 0.f, i1 = wl[1] > 0.f || wl[1] != wl[1] ? 1.f / wl[1] : 0.f;
    const uint32_t r0 = turn8x8(pack2<T>(w[0] * i0, w[1] * i1)), r1 = turn8x8(pack2<T>(w[2] * i0, w[3] * i1));
    const int c = (run % a.runs) * (8 * NT) + n * 8 + g;  // head g, elements 2t and 2t + 1
    if (c >= a.share) return;
    T* out = reinterpret_cast<T*>(a.o) + b * a.so_b + ((int64_t)(run / a.runs) * a.share + c) * a.so_h + d * 16 + 2 * t;
    if (a.o_even) {
      *reinterpret_cast<uint32_t*>(out) = r0;
      *reinterpret_cast<uint32_t*>(out + 8) = r1;
    } else {
      reinterpret_cast<uint16_t*>(out)[0] = (uint16_t)r0, reinterpret_cast<uint16_t*>(out)[1] = (uint16_t)(r0 >> 16);
      reinterpret_cast<uint16_t*>(out)[8] = (uint16_t)r1, reinterpret_cast<uint16_t*>(out)[9] = (uint16_t)(r1 >> 16);
    }
  };
  // PRE: leaves 16 elements from 16 * d on of run n's heads, and m and l, unscaled
  auto leave_out = [&](int b, int run, int n, int d, const float (&w)[4]) {
#pragma unroll
    for (int x = 0; x < 2; x++) {
      const int c = (run % a.runs) * (8 * NT) + n * 8 + 2 * t + x;
      if (c >= a.share) continue;
      float* at = a.own + 2 * a.own_rows + (((int64_t)(run / a.runs) * a.lanes + b) * a.share + c) * D + d * 16 + g;
      at[0] = w[x], at[8] = w[2 + x];
    }
  };
  auto leave_ml = [&](int b, int run, int n, const float (&mm)[2], const float (&ll)[2]) {
#pragma unroll
    for (int x = 0; x < 2; x++) {
      const int c = (run % a.runs) * (8 * NT) + n * 8 + 2 * t + x;
      if (c >= a.share) continue;
      float* at = a.own + ((int64_t)(run / a.runs) * a.lanes + b) * a.share + c;
      at[0] = mm[x], at[a.own_rows] = ll[x];
    }
  };
  auto put_lse = [&](int b, int run, const float (&wm)[NT][2], const float (&wl)[NT][2]) {
    if (!a.lse) return;
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int x = 0; x < 2; x++) {
        const int c = (run % a.runs) * (8 * NT) + n * 8 + 2 * t + x;
        if (c < a.share)
          a.lse[b * a.sl_b + (int64_t)(run / a.runs) * a.share + c] = (wm[n][x] + (log2f(wl[n][x]) - kLift<T>)) * kLn2;
      }
  };
  // lane and run whose units are shared with other CTAs: at this one's start and end
  struct Shared_out {
    bool some = false;
    int b, run;
    uint32_t seg0, tiles;
  } left0, left1;
  bool whole_start = at.tile == 0;
  bool from_u0 = true;  // the segment holds the range's first unit

  int get = 0;
  for (uint32_t u = u0; u < u1; u++) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    __syncwarp();
    copy_next(S % 2 == 0);
    const uint32_t kt = ring + get * kTile;
    get = get + 1 == S ? 0 : get + 1;
    const bool ok0 = ok_bits >> (2 * ((u - u0) & 7)) & 1u, ok1 = ok_bits >> (2 * ((u - u0) & 7) + 1) & 1u;

    // several sums, so that the instructions do not wait for one another
    constexpr int P = 4 / NT;
    float s[NT][4], sp[P][NT][4];
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int i = 0; i < P; i++) sp[i][n][0] = sp[i][n][1] = sp[i][n][2] = sp[i][n][3] = 0.f;
    {
      const int r = (lane & 7) + (lane >> 3 & 1) * 8;
#pragma unroll
      for (int k = 0; k < KS; k++) {
        uint32_t f[4];
        ldm4(f, kt + r * (D * 2) + (((2 * k + (lane >> 4)) ^ (r & 7)) * 16));
#pragma unroll
        for (int n = 0; n < NT; n++) mma16816<T>(sp[k % P][n], f[0], f[1], f[2], f[3], qf[n][k][0], qf[n][k][1]);
      }
    }
    constexpr bool kThird = std::is_same_v<T, __nv_bfloat16>;  // P's parts
    uint32_t hi[NT][2], lo[NT][2], last[NT][2];
#pragma unroll
    for (int n = 0; n < NT; n++) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        s[n][i] = sp[0][n][i];
#pragma unroll
        for (int j = 1; j < P; j++) s[n][i] += sp[j][n][i];
      }
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
      // (the difference first: it is 0 at most however large the scores are)
      auto weight = [&](float x, float ref) { return exp2a(kLift<T> != 0.f ? (x - ref) + kLift<T> : x - ref); };
      const float p0 = weight(s[n][0], top[0]), p1 = weight(s[n][1], top[1]);
      const float p2 = weight(s[n][2], top[0]), p3 = weight(s[n][3], top[1]);
      l[n][0] = l[n][0] * keep[0] + (p0 + p2);
      l[n][1] = l[n][1] * keep[1] + (p1 + p3);
      const uint32_t h0 = pack2<T>(p0, p1), h1 = pack2<T>(p2, p3);
      const float2 f0 = unpack2<T>(h0), f1 = unpack2<T>(h1);
      hi[n][0] = turn8x8(h0);
      hi[n][1] = turn8x8(h1);
      const uint32_t l0 = pack2<T>(p0 - f0.x, p1 - f0.y), l1 = pack2<T>(p2 - f1.x, p3 - f1.y);
      lo[n][0] = turn8x8(l0);
      lo[n][1] = turn8x8(l1);
      if (kThird) {
        const float2 g0 = unpack2<T>(l0), g1 = unpack2<T>(l1);
        last[n][0] = turn8x8(pack2<T>(p0 - f0.x - g0.x, p1 - f0.y - g0.y));
        last[n][1] = turn8x8(pack2<T>(p2 - f1.x - g1.x, p3 - f1.y - g1.y));
      }
#pragma unroll
      for (int d = 0; d < DT; d++) {
        o[n][d][0] *= keep[0];
        o[n][d][1] *= keep[1];
        o[n][d][2] *= keep[0];
        o[n][d][3] *= keep[1];
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    __syncwarp();
    copy_next(S % 2 == 1);
    const uint32_t vt = ring + get * kTile;
    get = get + 1 == S ? 0 : get + 1;
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
          if (kThird) mma16816<T>(o[n][d], f[0], f[1], f[2], f[3], last[n][0], last[n][1]);
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
          for (int w = 0; w < W; w++) top = fmaxf(top, xm[(w * 2) * (8 * NT) + col]);
          const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
          for (int w = 0; w < W; w++)
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
      // the others hand theirs to warps 0 and 1, two at a time, which then exchange
      // halves of the elements
#pragma unroll 1
      for (int from = 2; from < W; from += 2) {
        if (warp == from || warp == from + 1) {
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int d = 0; d < DT; d++)
              reinterpret_cast<float4*>(xo)[(((warp - from) * NT + n) * DT + d) * 32 + lane] =
                  make_float4(o[n][d][0], o[n][d][1], o[n][d][2], o[n][d][3]);
        }
        __syncthreads();
        if (warp < 2) {
          const bool last = from + 2 == W;
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int d = 0; d < DT; d++) {
              float4* at_xo = reinterpret_cast<float4*>(xo) + ((warp * NT + n) * DT + d) * 32 + lane;
              const float4 v = *at_xo;
              o[n][d][0] += v.x;
              o[n][d][1] += v.y;
              o[n][d][2] += v.z;
              o[n][d][3] += v.w;
              if (last && (d < DT / 2) != (warp == 0))
                *at_xo = make_float4(o[n][d][0], o[n][d][1], o[n][d][2], o[n][d][3]);
            }
        }
        __syncthreads();
      }
      const bool whole = whole_start && ends;
      if (warp < 2) {
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int e = 0; e < DT / 2; e++) {
            const int d = e + warp * (DT / 2);  // this warp's half
            const float4 v = reinterpret_cast<float4*>(xo)[(((1 - warp) * NT + n) * DT + d) * 32 + lane];
            float w[4] = {warp ? o[n][e + DT / 2][0] : o[n][e][0], warp ? o[n][e + DT / 2][1] : o[n][e][1],
                          warp ? o[n][e + DT / 2][2] : o[n][e][2], warp ? o[n][e + DT / 2][3] : o[n][e][3]};
            w[0] += v.x, w[1] += v.y, w[2] += v.z, w[3] += v.w;
            if (whole) {
              if (PRE)
                leave_out(at.b, at.run, n, d, w);
              else
                put_out(at.b, at.run, n, d, w, l[n]);
            } else {  // to the workspace; the last CTA adds up, below
              float* part = a.parts + ((int64_t)blockIdx.x * 2 + (from_u0 ? 0 : 1)) * kPartFloats;
              reinterpret_cast<float4*>(part + 2 * kColsMost)[(n * DT + d) * 32 + lane] = make_float4(w[0], w[1], w[2], w[3]);
            }
          }
        if (warp == 0 && g == 0) {
          if (whole) {
            if (PRE) {
#pragma unroll
              for (int n = 0; n < NT; n++) leave_ml(at.b, at.run, n, m[n], l[n]);
            } else {
              put_lse(at.b, at.run, m, l);
            }
          } else {
            float* part = a.parts + ((int64_t)blockIdx.x * 2 + (from_u0 ? 0 : 1)) * kPartFloats;
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
              for (int c = 0; c < 2; c++) {
                part[n * 8 + 2 * t + c] = m[n][c];
                part[kColsMost + n * 8 + 2 * t + c] = l[n][c];
              }
          }
        }
      }
      if (!whole) {
        Shared_out& w = from_u0 ? left0 : left1;
        w.some = true, w.b = at.b, w.run = at.run, w.seg0 = seg0, w.tiles = at.s.tiles;
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

  // ---- heads that are shared with other CTAs: the last one of them adds up, in CTA order
  if (!left0.some && !left1.some) {
    if (PRE) ops_begin();
    return;
  }
  if (warp < 2) __threadfence();
  __syncthreads();
  if (tid < 2) {
    const Shared_out& w = tid ? left1 : left0;
    s_last[tid] = 0;
    if (w.some) {
      const uint32_t c0 = cta_of(w.seg0), c1 = cta_of(w.seg0 + w.tiles - 1);
      const bool is_last = atomicAdd(a.counters + c0, 1u) == c1 - c0;
      if (is_last) {
        a.counters[c0] = 0;  // as the next call wants it
        __threadfence();
      }
      s_last[tid] = is_last;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < 2; i++) {
    if (!s_last[i]) continue;
    const Shared_out w = i ? left1 : left0;
    const uint32_t c0 = cta_of(w.seg0), c1 = cta_of(w.seg0 + w.tiles - 1);
    constexpr int E = DT / W;  // 16-element tiles of a warp
#pragma unroll
    for (int n = 0; n < NT; n++) {
      float mm[2] = {-INFINITY, -INFINITY}, ll[2] = {0.f, 0.f}, oo[E][4];
#pragma unroll
      for (int e = 0; e < E; e++) oo[e][0] = oo[e][1] = oo[e][2] = oo[e][3] = 0.f;
#pragma unroll 2
      for (uint32_t c = c0; c <= c1; c++) {
        const int which = c > c0 || first_of(c) == w.seg0 ? 0 : 1;
        const float* part = a.parts + ((int64_t)c * 2 + which) * kPartFloats;
        const float2 pm = __ldcg(reinterpret_cast<const float2*>(part + n * 8) + t);
        const float2 pl = __ldcg(reinterpret_cast<const float2*>(part + kColsMost + n * 8) + t);
        float4 v[E];
#pragma unroll
        for (int e = 0; e < E; e++)
          v[e] = __ldcg(reinterpret_cast<const float4*>(part + 2 * kColsMost) + (n * DT + warp * E + e) * 32 + lane);
        float keep[2], add[2];
#pragma unroll
        for (int x = 0; x < 2; x++) {
          const float one_m = x ? pm.y : pm.x, one_l = x ? pl.y : pl.x;
          const float now = fmaxf(mm[x], one_m), ref = now == -INFINITY ? 0.f : now;
          keep[x] = exp2a(mm[x] - ref);
          add[x] = exp2a(one_m - ref);
          mm[x] = now;
          ll[x] = ll[x] * keep[x] + one_l * add[x];
        }
#pragma unroll
        for (int e = 0; e < E; e++) {
          oo[e][0] = oo[e][0] * keep[0] + v[e].x * add[0];
          oo[e][1] = oo[e][1] * keep[1] + v[e].y * add[1];
          oo[e][2] = oo[e][2] * keep[0] + v[e].z * add[0];
          oo[e][3] = oo[e][3] * keep[1] + v[e].w * add[1];
        }
      }
#pragma unroll
      for (int e = 0; e < E; e++) {
        if (PRE)
          leave_out(w.b, w.run, n, warp * E + e, oo[e]);
        else
          put_out(w.b, w.run, n, warp * E + e, oo[e], ll);
      }
      if (PRE && warp == 0 && g == 0) leave_ml(w.b, w.run, n, mm, ll);
      m[n][0] = mm[0], m[n][1] = mm[1], l[n][0] = ll[0], l[n][1] = ll[1];
    }
    if (!PRE && warp == 0 && g == 0) put_lse(w.b, w.run, m, l);
  }
  if (PRE) ops_begin();
}


template <typename T, int D, int NT, bool PRE>
cudaError_t launch(const Args& a, int64_t most_units, cudaStream_t st) {
  auto* fn = attend_kernel<T, D, NT, PRE>;
  constexpr int smem = kSmem<D, NT>;
  static OpsOnce once;
  static int resident = 1;  // CTAs of a multiprocessor
  if (const int dev = ops_current(); !once(dev)) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int v = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, fn, kWarps<D> * 32, smem);
    if (e != cudaSuccess) return e;
    resident = v > 0 ? v : 1;
    once.set(dev);
  }
  int64_t grid = (int64_t)resident * ops_sm_count();
  if (grid > kMaxGrid) grid = kMaxGrid;
  if (grid > most_units) grid = most_units;
  return ops_launch(fn, (unsigned)grid, kWarps<D> * 32, smem, 0, st, a);
}

template <typename T, int D>
cudaError_t by_share(Args& a, int64_t tiles, cudaStream_t st) {
  if (a.share <= 8) {
    a.runs = 1;
    return a.own ? launch<T, D, 1, true>(a, tiles * a.hkv, st) : launch<T, D, 1, false>(a, tiles * a.hkv, st);
  }
  a.runs = (a.share + 15) / 16;
  const int64_t units = tiles * a.hkv * a.runs;
  return a.own ? launch<T, D, 2, true>(a, units, st) : launch<T, D, 2, false>(a, units, st);
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

extern "C" int wfst_attend_paged(const wfst_attend_args* r, void* stream) { return attend_behind(r, nullptr, stream); }

extern "C" int wfst_attend_size(int64_t* bytes) {
  if (!bytes) return api_fail(WFST_ERR_INVALID_ARG, "attend_size: NULL argument");
  *bytes = kCounterBytes + (int64_t)kMaxGrid * 2 * kPartFloats * 4;
  return WFST_OK;
}

int wfst::attend_behind(const wfst_attend_args* r, float* own, void* stream) {
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
  a.so_b = stride(r->o_stride[0], r->lanes), a.so_h = stride(r->o_stride[1], r->q_heads), a.sl_b = r->lse_stride;
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
  a.own = own;
  a.own_rows = ((int64_t)r->lanes * r->q_heads + 3) / 4 * 4;
  a.o_even = aligned(r->o, 4) && a.so_b % 2 == 0 && a.so_h % 2 == 0;
  int64_t most = (int64_t)r->table_width * r->page_size;
  if (a.window && (int64_t)a.window + a.sinks < most) most = (int64_t)a.window + a.sinks;
  const int64_t tiles = (int64_t)a.lanes * (most / kLeastUnit + 1);
  if (tiles * ((int64_t)a.hkv * ((a.share + 7) / 8)) > UINT32_MAX)
    return api_fail(WFST_ERR_INVALID_ARG, "attend_paged: lanes * kv_heads * tokens is too large");
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = r->dtype == WFST_F16 ? by_width<__half>(a, r->head_dim, tiles, st)
                                             : by_width<__nv_bfloat16>(a, r->head_dim, tiles, st);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "attend_paged launch");
}
