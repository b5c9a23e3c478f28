// wfst_prefix.cu — attention of one new token per lane behind a prefix that all
// lanes share.
//
//   lane b sees the prefix' tokens and then its own; for each query head
//   S_j = scale * q . k_j,  o = sum_j softmax(S)_j v_j,  lse = log sum_j exp S_j
//
// A pass has to read the prefix' keys and values once, 4 * D bytes per token and
// key-value head, for 4 * D flops per query head and lane: with R = lanes * (query
// heads to a key-value head) rows HBM bounds it up to some 200 rows, the tensor
// cores above.  So the prefix is a matrix product here: the R rows of a key-value
// head are the rows of S = Q K^T and O = P V on tcgen05.  Each CTA leaves the m, l
// and unscaled o of its share of the keys; the kernel of wfst_attend.cu attends to
// each lane's own tokens meanwhile and adds these parts to its own.
//
// A CTA takes 128 keys by 128 or 256 rows at a time (heads of 256: 64 by 128).  Four
// warps copy keys and values ahead into a ring (16 bytes a lane, since pages may end
// anywhere and lie in any order of strides), one issues the products, and a
// thread of four or eight more owns a row: it takes its row of S from tensor memory,
// where a row's maximum and sum need no exchange between threads, and puts P back
// in the same place as the operand of the second product.  There are two places for
// S, so that one is computed while the other one is exponentiated: two tiles of
// rows, or with up to 128 rows every other tile of keys (each with its own o, added
// up at the end), or, with heads of 256, whose o fills half of the tensor memory,
// the next tile of keys.
//
// o is rescaled only where a row's maximum has grown by more than 2^kSlack: the sum
// is the same with any reference.  P is held in two 16-bit parts, whose sum is off
// by at most 2^-16 of it (bf16; fp16: 2^-22), by two products into the same fp32
// sum.
//
// Work is split evenly whatever the sizes: the tiles of all heads and groups of rows are
// numbered through, and each CTA takes an equal range.
#include <cuda.h>

#include "wfst_ops.h"

namespace wfst {
namespace {

constexpr int kRows = 128;       // of a tile, one to a thread
constexpr int kMostGrid = 160;   // CTAs the workspace has room for: the multiprocessors of the chip
constexpr int kMaskRing = 8;     // tiles whose masks are kept, more than are ever in flight
constexpr uint32_t kNap = 20000, kSpins = 1u << 16;  // a wait sleeps so many ns at a time, and gives up after so many times
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 4.f;    // how far, in powers of two, a row's largest score may be above its reference
// fp16 has no exponents below 2^-24: P is held times 2^11, so that with kSlack it stays
// within 2^15 and what is lost is below 2^-35 of the largest weight; the parts that are
// left hold l and o times 2^15, as wfst_attend.cu does.
template <typename T>
constexpr float kLift = std::is_same_v<T, __half> ? 11.f : 0.f;
template <typename T>
constexpr float kLeft = std::is_same_v<T, __half> ? 16.f : 1.f;

// Keys of a tile; warpgroups that exponentiate; slots of the ring (keys or values of
// one tile each), as many as fit beside Q.
template <int D>
constexpr int kKeys = D == 256 ? 64 : 128;
template <int D>
constexpr int kGroups = D == 256 ? 1 : 2;
template <int D, int NQ>
constexpr int kSlots = D == 64 ? 8 : D == 256 ? 4 : NQ == 2 ? 4 : 5;
template <int D>
constexpr int kThreads = (kGroups<D> * 4 + 5) * 32;

struct Args {
  const void *q, *kc, *vc;
  const int32_t *table, *length;
  float* parts;
  int64_t sq_b, sq_h, ck_p, ck_s, ck_h, cv_p, cv_s, cv_h, room;
  int32_t lanes, hkv, share, groups, page, num_pages;
  uint32_t div_m, div_s, flip;  // flip: the signs of q, for a negative scale
  float scale2;                 // |scale| * log2(e)
};

// What lies behind Q and the ring in shared memory.
template <int S>
struct Control {
  uint64_t full[S], empty[S];          // a slot is filled, is free
  uint64_t s_full[2], p_full[2], pv[2];  // S is there, P is there, the second product is through
  uint64_t q_full, done;
  uint32_t masks[kMaskRing][4];        // keys of a tile that are seen
  float m[2][kRows], l[2][kRows];
  uint32_t tmem;
};
template <int D, int NQ>
constexpr int kSmem = 1024 + NQ * kRows * D * 2 + kSlots<D, NQ> * kKeys<D> * D * 2 + (int)sizeof(Control<kSlots<D, NQ>>);
static_assert(kSmem<64, 2> <= 232448 && kSmem<128, 1> <= 232448 && kSmem<128, 2> <= 232448 && kSmem<256, 1> <= 232448);

// ---- instructions

__device__ __forceinline__ bool test_bar(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
               : "=r"(done)
               : "r"(bar), "r"(parity)
               : "memory");
  return done;
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t i = 0; i < kSpins; i++) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kNap)
        : "memory");
    if (done) return true;
  }
  return false;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool elected() {
  uint32_t is;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(is));
  return is != 0;
}
// d (+)= a * b; a in shared memory, and in tensor memory
__device__ __forceinline__ void product_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// 32 columns of this warp's 32 lanes, when they are there
__device__ __forceinline__ void tmem_load(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// what plain stores and copies put into shared memory, for the tensor cores to see
__device__ __forceinline__ void smem_seen() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ float exp2a(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// Waits until all but the `open` youngest groups of this thread's copies have landed.
__device__ __forceinline__ void landed(int open) {
  switch (open) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
}

// Both operands' tiles lie in columns of 64 elements: rows of 128 bytes, whose 16-byte
// pieces are exchanged by row within 1024 bytes.  Q and K are read along the rows
// (groups of eight rows 1024 bytes apart), V across them (blocks of 64 elements
// `block` bytes apart, groups of eight keys 1024).
__device__ __forceinline__ uint64_t describe(uint32_t at, uint32_t block) {
  return (uint64_t)(at >> 4 & 0x3fffu) | (uint64_t)(block >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// NQ: tiles of rows of a CTA.
template <typename T, int D, int NQ>
__global__ void __launch_bounds__(kThreads<D>, 1) prefix_kernel(const Args a) {
  extern __shared__ unsigned char raw_smem[];
  constexpr int KT = kKeys<D>, G = kGroups<D>, S = kSlots<D, NQ>, kTile = KT * D * 2, kRowsAll = NQ * kRows;
  constexpr bool kTurns = NQ == 1;  // tiles of keys go to the two places of S in turn
  constexpr int kO = 2 * KT;        // tensor memory: two places of S, then o (two of them with G == 2)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* q_tile = raw_smem + ((1024 - ((uint32_t)__cvta_generic_to_shared(raw_smem) & 1023)) & 1023);
  unsigned char* ring = q_tile + kRowsAll * D * 2;
  auto& sh = *reinterpret_cast<Control<S>*>(ring + S * kTile);
  const uint32_t q_at = (uint32_t)__cvta_generic_to_shared(q_tile), ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  auto bar = [&](const uint64_t& b) { return (uint32_t)__cvta_generic_to_shared(&b); };

  ops_begin();
  ops_next();
  // ---- this CTA's tiles
  const int n = (int)max((int64_t)0, min((int64_t)*a.length, a.room));
  const uint32_t tiles = (n + KT - 1) / KT, units = tiles * a.hkv * a.groups;
  const uint32_t ctas = min(gridDim.x, units);
  if (blockIdx.x >= ctas) return;
  const uint32_t each = units / ctas, more = units - each * ctas;
  const uint32_t u0 = blockIdx.x * each + min(blockIdx.x, more), u1 = u0 + each + (blockIdx.x < more ? 1 : 0);

  if (tid == 0) {
    auto init = [&](const uint64_t& b, int count) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar(b)), "r"(count) : "memory");
    };
    for (int i = 0; i < S; i++) init(sh.full[i], 4), init(sh.empty[i], 1);
    for (int i = 0; i < 2; i++) init(sh.s_full[i], 2), init(sh.p_full[i], 4), init(sh.pv[i], 1);
    init(sh.q_full, 4 * G);
    init(sh.done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 4 * G + 4) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  const uint32_t tmem = sh.tmem;
  bool good = true;

  if (warp >= 4 * G && warp < 4 * G + 4) {
    // ---- copies: a warp takes a quarter of each tile's keys, in the order in which the tiles are needed
    constexpr int kMine = KT / 4, kLanes = D / 8, kAtOnce = 32 / kLanes;  // keys; lanes of a key, keys of an instruction
    const int w = warp - 4 * G;
    uint32_t issued = 0, told = 0;
    auto tell = [&]() {  // the oldest slot that is filled but not known to be
      landed((int)(issued - told) - 1);
      smem_seen();
      __syncwarp();
      if (lane == 0) arrive(bar(sh.full[told % S]));
      told++;
    };
    struct Key {
      int id, place;
    };
    auto look_up = [&](uint32_t tile) {
      Key k = {-1, 0};
      const int j = tile * KT + w * kMine + lane;
      if (lane < kMine && j < n) {
        const int pg = (int)(((uint64_t)(uint32_t)j * a.div_m) >> a.div_s);
        k.place = j - pg * a.page;
        k.id = ops_load(a.table + pg);
      }
      return k;
    };
    auto copy = [&](const Key& k, const void* pool, int64_t s_p, int64_t s_s, int64_t from) {
      const int slot = issued % S;
      if (issued >= S) {
        const uint32_t parity = (issued / S - 1) & 1;
        while (!__all_sync(0xffffffffu, test_bar(bar(sh.empty[slot]), parity))) {
          if (issued > told) {
            tell();
          } else {
            good = wait_bar(bar(sh.empty[slot]), parity);
            break;
          }
        }
        good = __all_sync(0xffffffffu, good);
        if (!good) return;
      }
      const bool seen = (uint32_t)k.id < (uint32_t)a.num_pages;
      const int64_t off = seen ? k.id * s_p + k.place * s_s + from : 0;
      const uint32_t some = __ballot_sync(0xffffffffu, seen);
      const uint32_t dst = ring_at + slot * kTile;
#pragma unroll 8
      for (int i = 0; i < kMine; i += kAtOnce) {
        const int mine = i + lane / kLanes, row = w * kMine + mine, piece = lane % kLanes;
        const int64_t o = __shfl_sync(0xffffffffu, off, mine);
        const int bytes = some >> mine & 1 ? 16 : 0;  // 0: sixteen zero bytes
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         dst + piece / 8 * (KT * 128) + row * 128 + ((piece % 8) ^ (row % 8)) * 16),
                     "l"(reinterpret_cast<const T*>(pool) + o + piece * 8), "r"(bytes)
                     : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      issued++;
      if (issued - told > 3) tell();
    };
    uint32_t count = 0;  // tiles whose keys have been copied
    for (uint32_t u = u0; u < u1 && good;) {
      const uint32_t group = u / tiles, t0 = u - group * tiles, some = min(tiles - t0, u1 - u);
      const int64_t head = group / a.groups;
      Key now[2], ahead = look_up(t0);
      auto keys = [&](uint32_t i) {
        const Key k = ahead;
        if (i % 2)
          now[1] = k;
        else
          now[0] = k;
        ahead = look_up(t0 + i + 1);
        const uint32_t ok = __ballot_sync(0xffffffffu, (uint32_t)k.id < (uint32_t)a.num_pages);
        copy(k, a.kc, a.ck_p, a.ck_s, head * a.ck_h);
        if (lane == 0) sh.masks[count % kMaskRing][w] = ok;
        count++;
      };
      constexpr uint32_t kLead = kTurns ? 2 : 1;
      for (uint32_t i = 0; i < kLead && i < some; i++) keys(i);
      for (uint32_t i = 0; i < some && good; i++) {
        copy(i % 2 ? now[1] : now[0], a.vc, a.cv_p, a.cv_s, head * a.cv_h);
        if (i + kLead < some) keys(i + kLead);
      }
      u += some;
    }
    while (good && issued > told) tell();
    landed(0);
  } else if (warp == 4 * G + 4) {
    // ---- products.  kind::f16: fp32 sums, 128 rows; Q K^T with N = KT, P V with N = D and V read across its rows
    constexpr uint32_t kType = std::is_same_v<T, __half> ? 0u : 1u;
    constexpr uint32_t kBase = 1u << 4 | kType << 7 | kType << 10 | (uint32_t)(kRows / 16) << 24;
    constexpr uint32_t kScores = kBase | (uint32_t)(KT / 8) << 17, kValues = kBase | (uint32_t)(D / 8) << 17 | 1u << 16;
    uint32_t taken = 0;          // slots of the ring, in order
    uint32_t s_used[2] = {0, 0};  // times either place has been used
    auto slot_in = [&]() {
      const int slot = taken % S;
      good = good && wait_bar(bar(sh.full[slot]), (taken / S) & 1);
      taken++;
      return slot;
    };
    auto scores = [&](int place, int q_tile_no, int slot, bool last) {
      __syncwarp();
      tmem_after();
      if (elected() && good) {
        const uint64_t q = describe(q_at + q_tile_no * (kRows * D * 2), 16), k = describe(ring_at + slot * kTile, 16);
#pragma unroll
        for (int s = 0; s < D / 16; s++)
          product_ss(tmem + place * KT, q + s / 4 * (kRows * 128 >> 4) + s % 4 * 2, k + s / 4 * (KT * 128 >> 4) + s % 4 * 2, kScores,
                     s != 0);
        commit(bar(sh.s_full[place]));
        arrive(bar(sh.s_full[place]));  // (what was seen before it, the tile's mask among it, is seen behind it)
        if (last) commit(bar(sh.empty[slot]));
      }
      __syncwarp();
    };
    auto values = [&](int place, int o_place, int slot, bool begins, bool last) {
      good = good && wait_bar(bar(sh.p_full[place]), s_used[place] & 1);
      s_used[place]++;
      __syncwarp();
      tmem_after();
      if (elected() && good) {
        const uint64_t v = describe(ring_at + slot * kTile, KT * 128);
#pragma unroll
        for (int s = 0; s < KT / 16; s++) {
          const uint32_t p = tmem + place * KT + s / 2 * 32 + s % 2 * 8;
          product_ts(tmem + kO + o_place * D, p, v + s * (2048 >> 4), kValues, !begins || s != 0);
          product_ts(tmem + kO + o_place * D, p + 16, v + s * (2048 >> 4), kValues, true);
        }
        commit(bar(sh.pv[place]));
        if (last) commit(bar(sh.empty[slot]));
      }
      __syncwarp();
    };
    // P lies where the next S goes
    auto through = [&](int place) { good = good && wait_bar(bar(sh.pv[place]), (s_used[place] - 1) & 1); };
    uint32_t segment = 0;
    for (uint32_t u = u0; u < u1;) {
      const uint32_t some = min(tiles - u % tiles, u1 - u);
      good = good && wait_bar(bar(sh.q_full), segment & 1);
      if (kTurns) {
        for (uint32_t i = 0; i < 2 && i < some; i++) scores(i, 0, slot_in(), true);
        for (uint32_t i = 0; i < some; i++) {
          const int place = i % 2;
          values(place, G == 2 ? place : 0, slot_in(), i < (uint32_t)G, true);
          if (i + 2 < some) {
            const int slot = slot_in();
            through(place);
            scores(place, 0, slot, true);
          }
        }
      } else {
        int slot = slot_in();
        scores(0, 0, slot, false);
        scores(1, 1, slot, true);
        for (uint32_t i = 0; i < some; i++) {
          const int v = slot_in();
          values(0, 0, v, i == 0, false);
          if (i + 1 < some) {
            slot = slot_in();
            through(0);
            scores(0, 0, slot, false);
          }
          values(1, 1, v, i == 0, true);
          if (i + 1 < some) {
            through(1);
            scores(1, 1, slot, true);
          }
        }
      }
      u += some;
      segment++;
    }
    // nothing may be on its way when its memory is given back, nor where a wait gave up
    __syncwarp();
    if (elected()) commit(bar(sh.done));
    __syncwarp();
    good = wait_bar(bar(sh.done), 0) && good;
  } else if (warp < 4 * G) {
    // ---- a row to each thread
    const int wg = warp / 4, row = tid % kRows;
    const uint32_t mine = tmem + (uint32_t)((warp % 4) * 32 << 16);  // this warp's lanes
    uint32_t used[2] = {0, 0}, count = 0;
    for (uint32_t u = u0; u < u1;) {
      const uint32_t group = u / tiles, some = min(tiles - u % tiles, u1 - u);
      const uint32_t head = group / a.groups, row0 = group % a.groups * kRowsAll, rows = (uint32_t)a.lanes * a.share;
      // ---- Q: each warpgroup its own tile of rows, or half of the one
      {
        constexpr int kPieces = D / 8, kStep = kTurns ? G * 128 : 128;
        for (int i = kTurns ? tid : tid % 128; i < kRows * kPieces; i += kStep) {
          const int r = i / kPieces + (kTurns ? 0 : wg * kRows), piece = i % kPieces;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (row0 + r < rows) {
            const uint32_t b = (row0 + r) / a.share, c = (row0 + r) - b * a.share;
            v = ops_load(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + b * a.sq_b +
                                                        ((int64_t)head * a.share + c) * a.sq_h + piece * 8));
            v.x ^= a.flip, v.y ^= a.flip, v.z ^= a.flip, v.w ^= a.flip;
          }
          *reinterpret_cast<uint4*>(q_tile + r / kRows * (kRows * D * 2) + piece / 8 * (kRows * 128) + r % kRows * 128 +
                                    ((piece % 8) ^ (r % 8)) * 16) = v;
        }
      }
      smem_seen();
      tmem_before();  // (the segment before: o has been read)
      __syncwarp();
      if (lane == 0) arrive(bar(sh.q_full));

      float ref = -INFINITY, l = 0.f;
      bool any = false;  // o holds something
      for (uint32_t i = kTurns && G == 2 ? wg : 0; i < some; i += kTurns && G == 2 ? 2 : 1) {
        const int place = kTurns ? i % 2 : wg;
        const uint32_t s_at = mine + place * KT, o_at = mine + kO + (G == 2 ? wg : 0) * D;
        good = good && wait_bar(bar(sh.s_full[place]), used[place] & 1);
        used[place]++;
        __syncwarp();
        tmem_after();
        uint32_t mask[KT / 32];
        bool whole = true;
        {
          const uint32_t* seen = sh.masks[(count + i) % kMaskRing];
#pragma unroll
          for (int c = 0; c < KT / 32; c++) {
            mask[c] = KT == 128 ? seen[c] : seen[2 * c] | seen[2 * c + 1] << 16;
            whole = whole && mask[c] == 0xffffffffu;
          }
        }
        uint32_t r[32];
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < KT / 32; c++) {
          tmem_load(r, s_at + c * 32);
          if (whole) {
#pragma unroll
            for (int j = 0; j < 32; j++) top = fmaxf(top, __uint_as_float(r[j]));
          } else {
#pragma unroll
            for (int j = 0; j < 32; j++)
              if (mask[c] >> j & 1) top = fmaxf(top, __uint_as_float(r[j]));
          }
        }
        const bool grows = top > ref && !((top - ref) * a.scale2 <= kSlack);
        if (__any_sync(0xffffffffu, grows)) {
          float keep = 1.f;
          if (grows) {
            keep = ref == -INFINITY ? 0.f : exp2a((ref - top) * a.scale2);
            ref = top;
            l *= keep;
          }
          if (any) {
            if (G == 1) {  // the product of the tile before may still be adding to o
              good = good && wait_bar(bar(sh.pv[place ^ 1]), (used[place ^ 1] - 1) & 1);
              __syncwarp();
              tmem_after();
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; c++) {
              tmem_load(r, o_at + c * 32);
#pragma unroll
              for (int j = 0; j < 32; j++) r[j] = __float_as_uint(__uint_as_float(r[j]) * keep);
              tmem_store(o_at + c * 32, r);
            }
            tmem_stored();
          }
        }
        any = true;
        const float from = ref == -INFINITY ? 0.f : ref;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < KT / 32; c++) {
          tmem_load(r, s_at + c * 32);
          uint32_t p[32];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float p0 = exp2a(fmaf(__uint_as_float(r[j]) - from, a.scale2, kLift<T>));
            float p1 = exp2a(fmaf(__uint_as_float(r[j + 1]) - from, a.scale2, kLift<T>));
            if (!whole) {
              p0 = mask[c] >> j & 1 ? p0 : 0.f;
              p1 = mask[c] >> (j + 1) & 1 ? p1 : 0.f;
            }
            sum[j / 2 % 2 * 2] += p0;
            sum[j / 2 % 2 * 2 + 1] += p1;
            const uint32_t hi = pack2<T>(p0, p1);
            const float2 f = unpack2<T>(hi);
            p[j / 2] = hi;
            p[16 + j / 2] = pack2<T>(p0 - f.x, p1 - f.y);
          }
          tmem_store(s_at + c * 32, p);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_stored();
        tmem_before();
        __syncwarp();
        if (lane == 0) arrive(bar(sh.p_full[place]));
      }
      if (kTurns && G == 2) used[wg ^ 1] += (some + wg) / 2;  // of the other warpgroup's place

      // ---- this CTA's part of the group
      float* part = a.parts + ((int64_t)blockIdx.x + group) * (kRowsAll * (2 + D));
      if (kTurns) {  // all products are through when the last one is
        good = good && wait_bar(bar(sh.pv[(some - 1) % 2]), (used[(some - 1) % 2] - 1) & 1);
      } else {
        good = good && wait_bar(bar(sh.pv[wg]), (used[wg] - 1) & 1);
      }
      __syncwarp();
      tmem_after();
      float4* out = reinterpret_cast<float4*>(part + 2 * kRowsAll);
      if (kTurns && G == 2) {
        sh.m[wg][row] = ref, sh.l[wg][row] = l;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const bool both = some > 1;
        const float m0 = sh.m[0][row], m1 = both ? sh.m[1][row] : -INFINITY, top = fmaxf(m0, m1);
        const float from = top == -INFINITY ? 0.f : top;
        const float f0 = m0 == -INFINITY ? 0.f : exp2a((m0 - from) * a.scale2) * kLeft<T>;
        const float f1 = m1 == -INFINITY ? 0.f : exp2a((m1 - from) * a.scale2) * kLeft<T>;
        if (wg == 0 && row0 + row < rows) {
          part[row] = good ? (top == -INFINITY ? top : top * a.scale2) : INFINITY;  // (makes NaN of what it is added to)
          part[kRowsAll + row] = sh.l[0][row] * f0 + (both ? sh.l[1][row] * f1 : 0.f);
        }
#pragma unroll 1
        for (int c = wg * (D / 64); c < (wg + 1) * (D / 64); c++) {
          uint32_t r[32], s[32];
          tmem_load(r, mine + kO + c * 32);
          if (both) tmem_load(s, mine + kO + D + c * 32);
#pragma unroll
          for (int j = 0; j < 32; j++)
            r[j] = __float_as_uint(__uint_as_float(r[j]) * f0 + (both ? __uint_as_float(s[j]) * f1 : 0.f));
          if (row0 + row < rows) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              out[(c * 8 + j / 4) * kRowsAll + row] = make_float4(__uint_as_float(r[j]), __uint_as_float(r[j + 1]),
                                                                  __uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]));
          }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");  // m and l may be written again
      } else {
        const int at = wg * kRows + row;
        if (row0 + at < rows) {
          part[at] = good ? (ref == -INFINITY ? ref : ref * a.scale2) : INFINITY;
          part[kRowsAll + at] = l * kLeft<T>;
        }
#pragma unroll 1
        for (int c = 0; c < D / 32; c++) {
          uint32_t r[32];
          tmem_load(r, mine + kO + wg * D + c * 32);
          if (row0 + at < rows) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              out[(c * 8 + j / 4) * kRowsAll + at] =
                  make_float4(__uint_as_float(r[j]) * kLeft<T>, __uint_as_float(r[j + 1]) * kLeft<T>,
                              __uint_as_float(r[j + 2]) * kLeft<T>, __uint_as_float(r[j + 3]) * kLeft<T>);
          }
        }
      }
      u += some;
      count += some;
    }
  }
  tmem_before();
  __syncthreads();
  if (warp == 4 * G + 4) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <typename T, int D, int NQ>
cudaError_t launch(const Args& a, int grid, cudaStream_t st) {
  auto* fn = prefix_kernel<T, D, NQ>;
  constexpr int smem = kSmem<D, NQ>;
  static OpsOnce once;
  if (const int dev = ops_current(); !once(dev)) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    once.set(dev);
  }
  return ops_launch(fn, dim3(grid), kThreads<D>, smem, 0, st, a);
}

template <typename T>
cudaError_t by_width(const Args& a, int d, int rows, int grid, cudaStream_t st) {
  if (d == 256) return launch<T, 256, 1>(a, grid, st);
  if (d == 128) return rows == kRows ? launch<T, 128, 1>(a, grid, st) : launch<T, 128, 2>(a, grid, st);
  return rows == kRows ? launch<T, 64, 1>(a, grid, st) : launch<T, 64, 2>(a, grid, st);
}

// Rows of a group: two tiles where one does not hold all of them, so that a key that
// has been copied is used twice.
int rows_of_group(int64_t rows, int d) { return d == 256 || rows <= kRows ? kRows : 2 * kRows; }

}  // namespace
}  // namespace wfst

using namespace wfst;

extern "C" int wfst_prefix_size(int32_t lanes, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t* bytes) {
  if (!bytes) return api_fail(WFST_ERR_INVALID_ARG, "prefix_size: NULL argument");
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return api_fail(WFST_ERR_INVALID_ARG, "prefix_size: head_dim must be 64, 128 or 256");
  if (lanes < 0 || q_heads < 0) return api_fail(WFST_ERR_INVALID_ARG, "prefix_size: counts must be >= 0");
  if (kv_heads < 1 || q_heads % kv_heads)
    return api_fail(WFST_ERR_INVALID_ARG, "prefix_size: q_heads must be a multiple of kv_heads");
  if ((int64_t)lanes * q_heads > INT32_MAX) return api_fail(WFST_ERR_INVALID_ARG, "prefix_size: too many heads");
  int64_t own;
  if (const int rc = wfst_attend_size(&own)) return rc;
  const int64_t rows = (int64_t)lanes * (q_heads / kv_heads), group = rows_of_group(rows, head_dim);
  const int64_t groups = (rows + group - 1) / group * kv_heads;
  *bytes = own + (kMostGrid + groups) * group * (2 + head_dim) * 4;
  return WFST_OK;
}

extern "C" int wfst_attend_prefix(const wfst_prefix_args* r, void* stream) {
  if (!r) return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: NULL argument");
  if (r->dtype != WFST_F16 && r->dtype != WFST_BF16) return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: bad dtype");
  int64_t bytes;
  if (const int rc = wfst_prefix_size(r->lanes, r->q_heads, r->kv_heads, r->head_dim, &bytes)) return rc;
  if (r->page_size < 1 || r->num_pages < 0 || r->table_width < 0 || r->prefix_width < 0)
    return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: page_size must be >= 1, num_pages and table widths >= 0");
  if ((int64_t)r->page_size * r->table_width > INT32_MAX - 1024 || (int64_t)r->page_size * r->prefix_width > INT32_MAX - 1024)
    return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: page_size times a table's width must stay below 2^31");
  if (!(r->scale == r->scale)) return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: scale must be a number");
  if (r->lanes == 0 || r->q_heads == 0) return WFST_OK;
  if (!r->q || !r->o || !r->prefix_length || !r->lengths || !r->workspace || (r->prefix_width && !r->prefix_table) ||
      (r->table_width && !r->table) || (r->num_pages && (!r->k_pages || !r->v_pages)))
    return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: NULL argument");
  for (const void* p : {r->q, r->k_pages, r->v_pages, (const void*)r->workspace})
    if (!aligned(p, 16)) return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: arrays must be 16-byte aligned");
  auto stride = [&](int64_t s, int64_t n) { return n > 1 ? s : 0; };
  const int64_t sq_b = stride(r->q_stride[0], r->lanes), sq_h = stride(r->q_stride[1], r->q_heads);
  const int64_t ck_p = stride(r->k_page_stride[0], r->num_pages), ck_s = stride(r->k_page_stride[1], r->page_size);
  const int64_t cv_p = stride(r->v_page_stride[0], r->num_pages), cv_s = stride(r->v_page_stride[1], r->page_size);
  const int64_t ck_h = stride(r->k_page_stride[2], r->kv_heads), cv_h = stride(r->v_page_stride[2], r->kv_heads);
  if ((sq_b | sq_h | ck_p | ck_s | ck_h | cv_p | cv_s | cv_h) & 7)
    return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: strides must be multiples of 8 elements");
  const int dev = ops_device(r->device, {r->q, r->k_pages, r->v_pages, r->prefix_table, r->prefix_length, r->table, r->lengths,
                                         r->o, r->lse, r->workspace});
  if (dev < 0) return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: every array must be device memory of one device");
  const int share = r->q_heads / r->kv_heads, rows = rows_of_group((int64_t)r->lanes * share, r->head_dim);
  const int64_t groups = ((int64_t)r->lanes * share + rows - 1) / rows, room = (int64_t)r->prefix_width * r->page_size;
  const int keys = r->head_dim == 256 ? kKeys<256> : kKeys<128>;
  const int64_t units = (room + keys - 1) / keys * groups * r->kv_heads;
  if (units > INT32_MAX) return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: lanes * heads * tokens is too large");
  int64_t own;
  if (const int rc = wfst_attend_size(&own)) return rc;
  OpsDevice guard(dev);
  if (guard.err != cudaSuccess) return api_cuda_fail(guard.err, "attend_prefix: device");
  PrefixParts pre = {};
  if (units) {
    Args a;
    a.q = r->q, a.kc = r->k_pages, a.vc = r->v_pages;
    a.table = r->prefix_table, a.length = r->prefix_length;
    a.parts = reinterpret_cast<float*>(static_cast<char*>(r->workspace) + own);
    a.sq_b = sq_b, a.sq_h = sq_h, a.ck_p = ck_p, a.ck_s = ck_s, a.ck_h = ck_h, a.cv_p = cv_p, a.cv_s = cv_s, a.cv_h = cv_h;
    a.room = room, a.lanes = r->lanes, a.hkv = r->kv_heads, a.share = share, a.groups = (int)groups;
    a.page = r->page_size, a.num_pages = r->num_pages;
    // key / page for key < 2^31: multiply by ceil(2^(31 + l) / page), l = ceil(log2 page)
    int l = 0;
    while ((int64_t)1 << l < r->page_size) l++;
    a.div_m = (uint32_t)((((uint64_t)1 << (31 + l)) + r->page_size - 1) / r->page_size);
    a.div_s = 31 + l;
    a.flip = r->scale < 0.f ? 0x80008000u : 0u;
    a.scale2 = (r->scale < 0.f ? -r->scale : r->scale) * kLog2e;
    int64_t grid = ops_sm_count();
    if (grid > kMostGrid) grid = kMostGrid;
    if (grid > units) grid = units;
    const cudaError_t e = r->dtype == WFST_F16 ? by_width<__half>(a, r->head_dim, rows, (int)grid, (cudaStream_t)stream)
                                               : by_width<__nv_bfloat16>(a, r->head_dim, rows, (int)grid, (cudaStream_t)stream);
    if (e != cudaSuccess) return api_cuda_fail(e, "attend_prefix launch");
    pre = {a.parts, r->prefix_length, room, keys, rows, (int)groups, (int)grid};
  }
  wfst_attend_args b = {};
  b.q = r->q, b.k_pages = r->k_pages, b.v_pages = r->v_pages, b.table = r->table, b.lengths = r->lengths;
  b.o = r->o, b.lse = r->lse, b.workspace = r->workspace;
  for (int i = 0; i < 2; i++) b.q_stride[i] = r->q_stride[i], b.o_stride[i] = r->o_stride[i];
  for (int i = 0; i < 3; i++) b.k_page_stride[i] = r->k_page_stride[i], b.v_page_stride[i] = r->v_page_stride[i];
  b.lse_stride = r->lse_stride, b.table_stride = r->table_stride;
  b.device = dev, b.dtype = r->dtype, b.lanes = r->lanes, b.q_heads = r->q_heads, b.kv_heads = r->kv_heads;
  b.head_dim = r->head_dim, b.table_width = r->table_width, b.num_pages = r->num_pages, b.page_size = r->page_size;
  b.scale = r->scale;
  return attend_behind(&b, units ? &pre : nullptr, stream);
}
