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
// head are the rows of S = Q K^T and O = P V on tcgen05.  Three kernels: this one
// leaves m, l and the unscaled o of each CTA's share of the keys; that of
// wfst_attend.cu does so for each lane's own tokens, and starts as this one's CTAs end;
// the last one puts them together.  (Put together at the end of the second one, whose
// CTAs take a lane and head after the other: 128 x 32767 241 us instead of 180.)
//
// A CTA takes tiles of keys by 128 or 256 rows.  Four warps copy keys and values ahead
// into a ring: in boxes of up to 32 keys by 64 elements where pages hold whole ones and
// all keys are there, otherwise 16 bytes a lane.  Two streams of tiles are under way at
// once, so that one's scores are exponentiated while the tensor cores work for the other:
// with more than 128 rows two tiles of rows, which share the keys that were copied, with
// up to 128 every other tile of keys, each with its own o.  A warp issues each stream's
// products, and a thread of four or eight warps owns a row: it takes its row of S from
// tensor memory, where the maximum and sum need no exchange between threads, 64
// scores at a time, and puts P in their place, as the operand of the second product.
// Heads of 256, whose o fills half of the tensor memory, have one stream.
//
// Tiles are of 128 keys where the copies bound it (up to 128 rows): S is computed once
// for either half's P.  With two tiles of rows they are of 64, and S is computed a tile
// ahead: 147 us became 130 with 64 x 16 rows of 32767 keys, but 16 x 4 of 131072 took 114
// instead of 101.
//
// o is rescaled only where a row's maximum has grown by more than 2^kSlack: the sum
// is the same with any reference.  P is held in two 16-bit parts, whose sum is off
// by at most 2^-16 of it (bf16; fp16: 2^-22), by two products into the same fp32
// sum.  (One part would be off by as much as o's own rounding; with a first part that is
// cut off instead of rounded, 2^-15, 128 x 32767 takes 180 us instead of 185.)
//
// Work is split evenly whatever the sizes: the tiles of all heads and groups of rows are
// numbered through, and each CTA takes an equal range.
//
// Heads of 128, bf16: 16 lanes with 32 query and 8 key-value heads behind 131072 tokens
// (0.54 GB) take 101 us, 5.5 TB/s; 128 lanes with 64 and 8 heads behind 32767, and their own
// 500 at most (0.27 GB), 186: this kernel 135, of which the tensor cores are busy for 108 at
// their measured rate, the lanes' own tokens 42, the joining 6; 64 lanes with 32 and 8
// heads behind 8192 43; 8 lanes with 16 and 16 heads of 64, fp16, behind 500 8.
#include <cuda.h>

#include <cfloat>

#include "wfst_ops.h"

namespace wfst {
namespace {

constexpr int kRows = 128;       // of a tile, one to a thread
constexpr int kMostGrid = 160;   // CTAs the workspace has room for: the multiprocessors of the chip
constexpr int kMaskRing = 16;    // tiles whose masks are kept, more than are ever in flight
constexpr uint32_t kNap = 20000, kSpins = 1u << 16;  // a wait sleeps so many ns at a time, and gives up after so many times
constexpr int kLooks = 200;      // before it sleeps at all: a warp that has gone to sleep wakes some 500 cycles late
constexpr float kLog2e = 1.4426950408889634f;
// How far, in powers of two, a row's largest score may be above its reference.  fp16
// has no exponents below 2^-24: P is held times 2^11, so that with kSlack it stays within
// 2^15 and what is lost is below 2^-35 of the largest weight; the parts that are left
// hold l and o times 2^15, as wfst_attend.cu does.
template <typename T>
constexpr float kSlack = std::is_same_v<T, __half> ? 4.f : 8.f;
template <typename T>
constexpr float kLift = std::is_same_v<T, __half> ? 11.f : 0.f;
template <typename T>
constexpr float kLeft = std::is_same_v<T, __half> ? 16.f : 1.f;

// Keys of a tile; warpgroups that exponentiate; slots of the ring (keys or values of
// one tile each), as many as fit beside Q.
template <int D, int NQ>
constexpr int kKeys = D == 256 || NQ == 2 ? 64 : 128;
template <int D>
constexpr int kGroups = D == 256 ? 1 : 2;
template <int D, int NQ>
constexpr int kSlots = D == 256 ? 4 : NQ == 2 ? 8 : 6;
template <int D>
constexpr int kThreads = (kGroups<D> * 5 + 4) * 32;

struct Args {
  const void *q, *kc, *vc;
  const int32_t *table, *length;
  float* parts;
  int64_t sq_b, sq_h, ck_p, ck_s, ck_h, cv_p, cv_s, cv_h, room;
  int32_t lanes, hkv, share, groups, page, num_pages;
  uint32_t div_m, div_s, flip;  // flip: the signs of q, for a negative scale
  float scale2;                 // |scale| * log2(e)
  int32_t box;                  // keys of a page that one copy takes; 0: the maps are not for use
};

// What lies behind Q and the ring in shared memory.
template <int S>
struct Control {
  uint64_t full[S], empty[S];  // a slot is filled, is free
  // of each stream's 128 columns S is in halves: S is there, P is there, the second product is through
  uint64_t s_full[2][2], p_full[2][2], pv[2][2];
  uint64_t q_full[2], done[2];   // of a stream: Q is there, all its products are through
  uint32_t masks[kMaskRing][4];  // keys of a tile that are seen, a quarter to a word
  uint32_t tmem;
};
template <int D, int NQ>
constexpr int kSmem = 1024 + NQ * kRows * D * 2 + kSlots<D, NQ> * kKeys<D, NQ> * D * 2 + (int)sizeof(Control<kSlots<D, NQ>>);
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
  for (int i = 0; i < kLooks; i++)
    if (test_bar(bar, parity)) return true;
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
__device__ __forceinline__ bool elected() {
  uint32_t is;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(is));
  return is != 0;
}
// a box of 64 elements by some keys of a page
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int element, int place, int head, int page,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(map), "r"(element), "r"(place), "r"(head), "r"(page), "r"(bar)
      : "memory");
}
// What the products' warp issues, by the one lane that `one` is not zero in.  The
// predicate is on the instruction and there is no branch around it: what the matrix
// instructions take has to be in registers that a warp has in common, and in a branch
// of one lane it is moved there for each of them, which takes longer than a product.
// The upper half of what describes an operand in shared memory: groups of eight rows
// 1024 bytes apart, 16-byte pieces exchanged within that.
constexpr uint32_t kUpper = 1024 >> 4 | 1u << 14 | 2u << 29;
// d (+)= a * b; a in shared memory, and in tensor memory
__device__ __forceinline__ void product_ss(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p, q;\n.reg .b64 x, y;\nsetp.ne.u32 p, %4, 0;\nsetp.ne.u32 q, %6, 0;\n"
      "mov.b64 x, {%1, %5};\nmov.b64 y, {%2, %5};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kUpper), "r"(one)
      : "memory");
}
__device__ __forceinline__ void product_ts(uint32_t one, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p, q;\n.reg .b64 y;\nsetp.ne.u32 p, %4, 0;\nsetp.ne.u32 q, %6, 0;\n"
      "mov.b64 y, {%2, %5};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kUpper), "r"(one)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.u32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar),
      "r"(one)
      : "memory");
}
__device__ __forceinline__ void arrive(uint32_t one, uint32_t bar) {
  asm volatile("{\n.reg .pred q;\nsetp.ne.u32 q, %1, 0;\n@q mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(bar), "r"(one)
               : "memory");
}
// 32 columns of this warp's 32 lanes: asked for, and there (the registers go through
// the wait, so that nothing that uses them is moved before it)
__device__ __forceinline__ void tmem_ask(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_there(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t (&r)[32], uint32_t at) {
  tmem_ask(r, at);
  tmem_there(r);
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
// 16 columns
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
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
// Two fp32 numbers at once.
struct Two {
  uint64_t v;
  __device__ __forceinline__ Two() {}
  __device__ __forceinline__ Two(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
  __device__ __forceinline__ float2 get() const {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
  }
};
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// A value that all lanes of a warp have, so that the compiler knows it: a reduction's
// result is in a register that the warp has in common.
__device__ __forceinline__ uint32_t same(uint32_t v) { return __reduce_or_sync(0xffffffffu, v); }

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
__device__ __forceinline__ uint32_t describe(uint32_t at, uint32_t block) { return (at >> 4 & 0x3fffu) | (block >> 4) << 16; }

// NQ: tiles of rows of a CTA.
template <typename T, int D, int NQ>
__global__ void __launch_bounds__(kThreads<D>, 1)
    prefix_kernel(const Args a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ unsigned char raw_smem[];
  constexpr int KT = kKeys<D, NQ>, G = kGroups<D>, S = kSlots<D, NQ>, kTile = KT * D * 2, kRowsAll = NQ * kRows;
  // G streams of scores: of a tile of rows each, or of every other tile of keys (kTurns).
  // A stream has 128 columns of tensor memory for S, which are exponentiated 64 at a
  // time: the halves of a tile of keys (H == 2), or two tiles (H == 1).  P takes the place
  // of S.  o lies behind them.
  constexpr bool kTurns = NQ == 1 && G == 2;
  constexpr int H = KT / 64, kO = 256;
  // Slots of the ring go round for both streams together, or, with kTurns, for either by
  // itself; a tile's keys are item 2 t of it, its values item 2 t + 1.
  constexpr int R = kTurns ? S / 2 : S;
  const int tid = threadIdx.x, lane = tid & 31, warp = (int)same(tid >> 5);
  unsigned char* q_tile = raw_smem + ((1024 - ((uint32_t)__cvta_generic_to_shared(raw_smem) & 1023)) & 1023);
  unsigned char* ring = q_tile + kRowsAll * D * 2;
  auto& sh = *reinterpret_cast<Control<S>*>(ring + S * kTile);
  const uint32_t q_at = (uint32_t)__cvta_generic_to_shared(q_tile), ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  auto bar = [&](const uint64_t& b) { return (uint32_t)__cvta_generic_to_shared(&b); };

  ops_begin();
  ops_next();
  // ---- this CTA's tiles
  const int n = (int)same((uint32_t)max((int64_t)0, min((int64_t)*a.length, a.room)));
  const uint32_t tiles = (n + KT - 1) / KT, units = tiles * a.hkv * a.groups;
  const uint32_t ctas = min(gridDim.x, units);
  if (blockIdx.x >= ctas) return;
  const uint32_t each = units / ctas, more = units - each * ctas;
  const uint32_t u0 = blockIdx.x * each + min(blockIdx.x, more), u1 = u0 + each + (blockIdx.x < more ? 1 : 0);

  if (tid == 0) {
    auto init = [&](const uint64_t& b, int count) {
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar(b)), "r"(count) : "memory");
    };
    for (int i = 0; i < S; i++) init(sh.full[i], 4), init(sh.empty[i], NQ);
    for (int i = 0; i < 4; i++) init(sh.s_full[i / 2][i % 2], 2), init(sh.p_full[i / 2][i % 2], 4), init(sh.pv[i / 2][i % 2], 1);
    for (int i = 0; i < G; i++) init(sh.q_full[i], kTurns ? 8 : 4), init(sh.done[i], 1);
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
  const uint32_t tmem = same(sh.tmem);
  bool good = true;

  if (warp >= 4 * G && warp < 4 * G + 4) {
    // ---- copies: a warp takes a quarter of each tile's keys, in the order in which the tiles are needed
    constexpr int kMine = KT / 4, kLanes = D / 8, kAtOnce = 32 / kLanes;  // keys; lanes of a key, keys of an instruction
    const int w = warp - 4 * G;
    uint32_t pending[4] = {}, count = 0;  // barriers of the slots that are filled but not known to be, oldest first
    auto tell = [&]() {
      landed((int)count - 1);
      smem_seen();
      __syncwarp();
      if (lane == 0) arrive(1, pending[0]);
#pragma unroll
      for (int i = 0; i < 3; i++) pending[i] = pending[i + 1];
      count--;
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
    // A warp's keys that are all there come in boxes, if pages hold whole ones; the others one by one.
    auto copy = [&](int ring_no, uint32_t item, const Key& k, const CUtensorMap* map, int head, const void* pool, int64_t s_p,
                    int64_t s_s, int64_t s_h) {
      const int slot = ring_no * R + item % R;
      const bool seen = (uint32_t)k.id < (uint32_t)a.num_pages;
      const int64_t off = seen ? k.id * s_p + k.place * s_s + head * s_h : 0;
      const uint32_t some = __ballot_sync(0xffffffffu, seen), full = bar(sh.full[slot]), dst = ring_at + slot * kTile;
      if (a.box && some == 0xffffffffu >> (32 - kMine)) {
        if (lane == 0)
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full), "n"(kMine * D * 2) : "memory");
        __syncwarp();
        const int from = lane / (D / 64) * a.box, block = lane % (D / 64);
        const int id = __shfl_sync(0xffffffffu, k.id, from % 32), place = __shfl_sync(0xffffffffu, k.place, from % 32);
        if (from < kMine)
          copy_box(dst + block * (KT * 128) + (w * kMine + from) * 128, map, block * 64, place, head, id, full);
        return;
      }
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
      if (count == 0) pending[0] = full;
      if (count == 1) pending[1] = full;
      if (count == 2) pending[2] = full;
      if (count == 3) pending[3] = full;
      if (++count == 4) tell();
    };
    // waits for the slot of an item
    auto room = [&](int ring_no, uint32_t item) {
      if (item < (uint32_t)R || !good) return;
      const uint32_t free = bar(sh.empty[ring_no * R + item % R]), parity = (item / R - 1) & 1;
      while (!__all_sync(0xffffffffu, test_bar(free, parity))) {
        if (count) {
          tell();
        } else {
          good = wait_bar(free, parity);
          break;
        }
      }
      good = __all_sync(0xffffffffu, good);
    };
    uint32_t items[2] = {0, 0}, tile_no = 0;  // of either ring; all tiles
    for (uint32_t u = u0; u < u1 && good;) {
      const uint32_t group = u / tiles, t0 = u - group * tiles, some = min(tiles - t0, u1 - u);
      const int head = group / a.groups;
      Key ahead = look_up(t0);
      for (uint32_t i = 0; i < some && good; i++, tile_no++) {
        const int r = kTurns ? i % 2 : 0;
        const uint32_t item = r ? items[1] : items[0];
        const Key k = ahead;
        if (i + 1 < some) ahead = look_up(t0 + i + 1);
        const uint32_t seen = __ballot_sync(0xffffffffu, (uint32_t)k.id < (uint32_t)a.num_pages);
        room(r, item);
        if (!good) break;
        if (lane == 0) sh.masks[tile_no % kMaskRing][w] = seen;  // (the slot is free, and what went with its tile before it)
        copy(r, item, k, &k_map, head, a.kc, a.ck_p, a.ck_s, a.ck_h);
        room(r, item + 1);
        if (good) copy(r, item + 1, k, &v_map, head, a.vc, a.cv_p, a.cv_s, a.cv_h);
        (r ? items[1] : items[0]) += good ? 2 : 1;
      }
      u += some;
    }
    while (count) tell();
    // no box may be on its way when the CTA ends, nor where a wait gave up
#pragma unroll
    for (int r = 0; r < (kTurns ? 2 : 1); r++)
      for (uint32_t i = items[r] > (uint32_t)R ? items[r] - R : 0; i < items[r]; i++)
        if (!wait_bar(bar(sh.full[r * R + i % R]), i / R & 1)) break;
  } else if (warp >= 4 * G + 4) {
    // ---- products, a warp to each stream.  kind::f16: fp32 sums, 128 rows; Q K^T with N = KT, P V with N = D and
    // V read across its rows
    constexpr uint32_t kType = std::is_same_v<T, __half> ? 0u : 1u;
    constexpr uint32_t kBase = 1u << 4 | kType << 7 | kType << 10 | (uint32_t)(kRows / 16) << 24;
    constexpr uint32_t kScores = kBase | (uint32_t)(KT / 8) << 17, kValues = kBase | (uint32_t)(D / 8) << 17 | 1u << 16;
    const uint32_t one = elected();
    const int j = G == 2 ? warp - (4 * G + 4) : 0, ring_no = kTurns ? j : 0;
    // items of the ring, tiles that have been through the first product, halves (H == 2) or tiles through the second one
    uint32_t items = 0, scored = 0, summed = 0;
    auto slot_in = [&](uint32_t item) {
      const int slot = ring_no * R + item % R;
      good = good && wait_bar(bar(sh.full[slot]), item / R & 1);
      return slot;
    };
    // S of a tile, where P of the one before (H == 1: before that) was
    auto scores = [&](uint32_t item) {
      const int slot = slot_in(item);
      const uint32_t k = scored++, place = H == 2 ? 0 : k & 1;
      if (k >= 3 - H) good = good && wait_bar(bar(sh.pv[j][H == 2 ? 1 : place]), (H == 2 ? k - 1 : (k - 2) >> 1) & 1);
      good = __all_sync(0xffffffffu, good);
      if (!good) return;
      tmem_after();
      const uint32_t q = same(describe(q_at + (kTurns ? 0 : j) * (kRows * D * 2), 16));
      const uint32_t key = same(describe(ring_at + slot * kTile, 16));
      const uint32_t d = same(tmem + j * 128 + place * 64);
#pragma unroll
      for (int s = 0; s < D / 16; s++)
        product_ss(one, d, q + s / 4 * (kRows * 128 >> 4) + s % 4 * 2, key + s / 4 * (KT * 128 >> 4) + s % 4 * 2, kScores, s != 0);
      commit(one, bar(sh.s_full[j][place]));
      arrive(one, bar(sh.s_full[j][place]));  // (what was seen before it, the tile's mask among it, is seen behind it)
      commit(one, bar(sh.empty[slot]));
    };
    // and its P V
    auto values = [&](uint32_t item, bool begins) {
      const int slot = slot_in(item);
#pragma unroll 1
      for (int h = 0; h < H; h++) {
        const uint32_t m = summed++, x = m & 1;
        good = good && wait_bar(bar(sh.p_full[j][x]), m >> 1 & 1);
        good = __all_sync(0xffffffffu, good);
        if (!good) continue;
        tmem_after();
        const uint32_t v = same(describe(ring_at + slot * kTile + h * (64 * 128), KT * 128)), p = same(tmem + j * 128 + x * 64);
        const uint32_t d = same(tmem + kO + j * D);
#pragma unroll
        for (int s = 0; s < 4; s++) {
          product_ts(one, d, p + s * 16, v + s * (2048 >> 4), kValues, !begins || h || s);
          product_ts(one, d, p + s * 16 + 8, v + s * (2048 >> 4), kValues, true);
        }
        commit(one, bar(sh.pv[j][x]));
        if (h == H - 1) commit(one, bar(sh.empty[slot]));
      }
    };
    uint32_t segment = 0;  // those that the stream has a part in
    for (uint32_t u = u0; u < u1;) {
      const uint32_t some = min(tiles - u % tiles, u1 - u), steps = kTurns ? (some + 1 - j) / 2 : some;
      u += some;
      if (steps == 0) continue;
      good = good && wait_bar(bar(sh.q_full[j]), segment++ & 1);
      constexpr uint32_t kAhead = 3 - H;
      for (uint32_t i = 0; i < kAhead && i < steps; i++) scores(items + 2 * i);
      for (uint32_t i = 0; i < steps; i++) {
        values(items + 2 * i + 1, i == 0);
        if (i + kAhead < steps) scores(items + 2 * (i + kAhead));
      }
      items += 2 * steps;
    }
    // nothing may be on its way when its memory is given back, nor where a wait gave up
    commit(one, bar(sh.done[j]));
    good = wait_bar(bar(sh.done[j]), 0) && good;
  } else if (warp < 4 * G) {
    // ---- a row to each thread
    const int wg = warp / 4, row = tid % kRows;
    const uint32_t mine = tmem + (uint32_t)((warp % 4) * 32 << 16);  // this warp's lanes
    uint32_t used = 0, count = 0;  // tiles of the stream, and of the CTA before this segment's
    for (uint32_t u = u0; u < u1;) {
      const uint32_t group = u / tiles, some = min(tiles - u % tiles, u1 - u);
      const uint32_t head = group / a.groups, row0 = group % a.groups * kRowsAll, rows = (uint32_t)a.lanes * a.share;
      // ---- Q: each warpgroup its own tile of rows, or half of the one
      {
        constexpr int kPieces = D / 8, kStep = NQ == 1 ? G * 128 : 128, kEach = kRows * kPieces / kStep,
                      kBatch = kEach < 16 ? kEach : 16, kDown = kStep / kPieces;  // a thread's next piece is kDown rows below
        static_assert(kStep % kPieces == 0 && kEach % kBatch == 0);
        const int t0 = NQ == 1 ? tid : tid % 128, piece = t0 % kPieces;
        int r = t0 / kPieces;
        const uint32_t first = row0 + r + (NQ == 1 ? 0 : wg * kRows), down_b = kDown / a.share, down_c = kDown - down_b * a.share;
        uint32_t b = first / a.share, c = first - b * a.share;
        const T* q = reinterpret_cast<const T*>(a.q) + (int64_t)head * a.share * a.sq_h + piece * 8;
        unsigned char* to = q_tile + (NQ == 1 ? 0 : wg) * (kRows * D * 2) + piece / 8 * (kRows * 128);
#pragma unroll 1
        for (int n = 0; n < kEach; n += kBatch) {
          uint4 v[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; j++) {
            v[j] = make_uint4(0, 0, 0, 0);
            if (b < (uint32_t)a.lanes) v[j] = ops_load(reinterpret_cast<const uint4*>(q + b * a.sq_b + c * a.sq_h));
            b += down_b, c += down_c;
            if (c >= (uint32_t)a.share) c -= a.share, b++;
          }
#pragma unroll
          for (int j = 0; j < kBatch; j++, r += kDown) {
            v[j].x ^= a.flip, v[j].y ^= a.flip, v[j].z ^= a.flip, v[j].w ^= a.flip;
            *reinterpret_cast<uint4*>(to + r * 128 + ((piece % 8) ^ (r % 8)) * 16) = v[j];
          }
        }
      }
      smem_seen();
      tmem_before();  // (the segment before: o has been read)
      __syncwarp();
      // (each stream that has something to do is told, by all that have a part in its Q)
#pragma unroll
      for (int j = 0; j < G; j++)
        if (lane == 0 && (kTurns ? some > (uint32_t)j : j == wg)) arrive(1, bar(sh.q_full[j]));

      float ref = -INFINITY, l = 0.f;
      bool any = false;  // o holds something
      for (uint32_t i = kTurns ? wg : 0; i < some; i += kTurns ? 2 : 1) {
        const uint32_t k = used++;
        good = good && wait_bar(bar(sh.s_full[wg][H == 2 ? 0 : k & 1]), (H == 2 ? k : k >> 1) & 1);
#pragma unroll 1
        for (int h = 0; h < H; h++) {
          const uint32_t part = k * H + h, x = part & 1, s_at = mine + wg * 128 + x * 64, o_at = mine + kO + wg * D;
          __syncwarp();
          tmem_after();
          const uint32_t* seen = sh.masks[(count + i) % kMaskRing];
          uint32_t r[2][32];  // the scores; -inf where the key is not seen
          tmem_ask(r[0], s_at);
          tmem_ask(r[1], s_at + 32);
          tmem_there(r[0]);
          tmem_there(r[1]);
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 2; c++) {
            const uint32_t mask = H == 2 ? seen[2 * h + c] : seen[2 * c] | seen[2 * c + 1] << 16;
            if (mask != 0xffffffffu) {
#pragma unroll
              for (int j = 0; j < 32; j++)
                if (!(mask >> j & 1)) r[c][j] = 0xff800000u;
            }
#pragma unroll
            for (int j = 0; j < 32; j++) tops[j % 4] = fmaxf(tops[j % 4], __uint_as_float(r[c][j]));
          }
          const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
          const bool grows = top > ref && !((top - ref) * a.scale2 <= kSlack<T>);
          if (__any_sync(0xffffffffu, grows)) {
            float keep = 1.f;
            if (grows) {
              keep = ref == -INFINITY ? 0.f : exp2a((ref - top) * a.scale2);
              ref = top;
              l *= keep;
            }
            if (any) {
              // the product of the tile before may still be adding to o
              good = good && wait_bar(bar(sh.pv[wg][x ^ 1]), (part - 1) >> 1 & 1);
              __syncwarp();
              tmem_after();
#pragma unroll 1
              for (int c = 0; c < D / 32; c++) {
                uint32_t v[32];
                tmem_load(v, o_at + c * 32);
#pragma unroll
                for (int j = 0; j < 32; j++) v[j] = __float_as_uint(__uint_as_float(v[j]) * keep);
                tmem_store(o_at + c * 32, v);
              }
              tmem_stored();
            }
          }
          any = true;
          const float from = ref == -INFINITY ? 0.f : ref;
          const Two less(-from, -from), by(a.scale2, a.scale2), lift(kLift<T>, kLift<T>), minus(-1.f, -1.f);
          Two sum[2] = {Two(0.f, 0.f), Two(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 4; c++) {  // 16 keys: eight columns of first parts, eight of the rests
            uint32_t p[16];
#pragma unroll
            for (int j = 0; j < 8; j++) {
              const uint32_t* x = &r[c / 2][c % 2 * 16 + 2 * j];
              const float2 y = fma2(add2(Two(__uint_as_float(x[0]), __uint_as_float(x[1])), less), by, lift).get();
              const float p0 = exp2a(y.x), p1 = exp2a(y.y);
              const Two both(p0, p1);
              sum[j % 2] = add2(sum[j % 2], both);
              p[j] = pack2<T>(p0, p1);
              const float2 f = unpack2<T>(p[j]);
              const float2 rest = fma2(Two(f.x, f.y), minus, both).get();
              p[8 + j] = pack2<T>(rest.x, rest.y);
            }
            tmem_store(s_at + c * 16, p);
          }
          const float2 s0 = sum[0].get(), s1 = sum[1].get();
          l += (s0.x + s0.y) + (s1.x + s1.y);
          tmem_stored();
          tmem_before();
          __syncwarp();
          if (lane == 0) arrive(1, bar(sh.p_full[wg][x]));
        }
      }

      // ---- this CTA's part of the group
      float* part = a.parts + ((int64_t)blockIdx.x + group) * (kRowsAll * (2 + D));
      if (used) {  // a stream's products are through when its last one is
        const uint32_t last = used * H - 1;
        good = good && wait_bar(bar(sh.pv[wg][last & 1]), last >> 1 & 1);
      }
      if (kTurns) {  // here both streams' have to be
        __syncwarp();
        tmem_after();
        tmem_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
      }
      __syncwarp();
      tmem_after();
      float4* out = reinterpret_cast<float4*>(part + 2 * kRowsAll);
      if (kTurns) {
        float* const ml = reinterpret_cast<float*>(q_tile);  // (Q is not needed any more)
        ml[wg * 256 + row] = ref, ml[wg * 256 + 128 + row] = l;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const bool both = some > 1;
        const float m0 = ml[row], m1 = both ? ml[256 + row] : -INFINITY, top = fmaxf(m0, m1);
        const float from = top == -INFINITY ? 0.f : top;
        const float f0 = m0 == -INFINITY ? 0.f : exp2a((m0 - from) * a.scale2) * kLeft<T>;
        const float f1 = m1 == -INFINITY ? 0.f : exp2a((m1 - from) * a.scale2) * kLeft<T>;
        if (wg == 0 && row0 + row < rows) {
          part[row] = good ? (top == -INFINITY ? top : top * a.scale2) : INFINITY;  // (makes NaN of what it is added to)
          part[kRowsAll + row] = ml[128 + row] * f0 + (both ? ml[384 + row] * f1 : 0.f);
        }
#pragma unroll 1
        for (int c = wg * (D / 64); c < (wg + 1) * (D / 64); c++) {
          uint32_t r[32];
          float v[32];
          tmem_load(r, mine + kO + c * 32);
#pragma unroll
          for (int j = 0; j < 32; j++) v[j] = __uint_as_float(r[j]) * f0;
          if (both) {
            tmem_load(r, mine + kO + D + c * 32);
#pragma unroll
            for (int j = 0; j < 32; j++) v[j] += __uint_as_float(r[j]) * f1;
          }
          if (row0 + row < rows) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              out[(c * 8 + j / 4) * kRowsAll + row] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");  // Q may be written again
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
cudaError_t launch(const Args& a, const CUtensorMap (&maps)[2], int grid, cudaStream_t st) {
  auto* fn = prefix_kernel<T, D, NQ>;
  constexpr int smem = kSmem<D, NQ>;
  static OpsOnce once;
  if (const int dev = ops_current(); !once(dev)) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    once.set(dev);
  }
  return ops_launch(fn, dim3(grid), kThreads<D>, smem, 0, st, a, maps[0], maps[1]);
}

template <typename T>
cudaError_t by_width(const Args& a, const CUtensorMap (&maps)[2], int d, int rows, int grid, cudaStream_t st) {
  if (d == 256) return launch<T, 256, 1>(a, maps, grid, st);
  if (d == 128) return rows == kRows ? launch<T, 128, 1>(a, maps, grid, st) : launch<T, 128, 2>(a, maps, grid, st);
  return rows == kRows ? launch<T, 64, 1>(a, maps, grid, st) : launch<T, 64, 2>(a, maps, grid, st);
}

// The pool as the copies of boxes want it: (element, place, head, page), in any order of strides.
bool map_pool(CUtensorMap* map, CUtensorMapDataType type, const void* pool, int d, const Args& a, int64_t s_s, int64_t s_h,
              int64_t s_p) {
  static const auto encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult how;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &how) != cudaSuccess)
      fn = nullptr;
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(fn);
  }();
  const cuuint64_t size[4] = {(cuuint64_t)d, (cuuint64_t)a.page, (cuuint64_t)a.hkv, (cuuint64_t)a.num_pages};
  cuuint64_t stride[3];
  const int64_t s[3] = {s_s, s_h, s_p};
  for (int i = 0; i < 3; i++) {
    if (size[i + 1] > 1 && (s[i] <= 0 || s[i] >= (int64_t)1 << 38)) return false;
    stride[i] = size[i + 1] > 1 ? (cuuint64_t)s[i] * 2 : (cuuint64_t)d * 2;  // (along one entry, any)
  }
  const cuuint32_t box[4] = {64, (cuuint32_t)a.box, 1, 1}, step[4] = {1, 1, 1, 1};
  return encode && encode(map, type, 4, const_cast<void*>(pool), size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---- the parts put together
//
// A CTA takes eight rows of a key-value head and 4 Q elements of them, a thread four elements
// of one: with eight neighbours of a group the parts' 128 bytes.  Where that leaves threads, as
// many share a head's parts, whose sums are added up in order.
constexpr int kJoinRows = 8, kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
struct Join {
  const float *parts, *own;
  const int32_t* length;
  void* o;
  float* lse;
  int64_t so_b, so_h, sl_b, room, own_rows;
  int32_t hkv, share, rows, keys, group, groups, grid, o_even;  // rows: of a key-value head; group: rows of one
};
template <typename T, int D, int Q>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Join a) {
  constexpr int kSplit = kJoinThreads / kJoinRows / Q;
  __shared__ float ms[kMostGrid + 1][kJoinRows], ls[kMostGrid + 1][kJoinRows];
  __shared__ float tops[kJoinWarps][kJoinRows], sums[kJoinWarps][kJoinRows];
  __shared__ float4 more[kSplit][kJoinRows * Q];  // (the first of them is not used)
  constexpr int kSide = kJoinThreads / kJoinRows;
  const int head = blockIdx.y, side = threadIdx.x / kJoinRows, r = threadIdx.x % kJoinRows;
  const int row = min(blockIdx.x * kJoinRows + r, (uint32_t)a.rows - 1);  // (one past the end does the last one's work again)
  // (the length was there before the kernels that this one waits for)
  const uint32_t tiles = (uint32_t)((max((int64_t)0, min((int64_t)*a.length, a.room)) + a.keys - 1) / a.keys);
  const uint32_t units = tiles * a.hkv * a.groups, ctas = min((uint32_t)a.grid, units);
  const uint32_t group = head * a.groups + row / a.group, at = row % a.group;
  uint32_t first = 0, count = 0;  // CTAs that have a part of the group
  if (units) {
    const uint32_t each = units / ctas, more = units - each * ctas;
    auto owner = [&](uint32_t u) {
      const uint32_t big = more * (each + 1);
      return u < big ? u / (each + 1) : more + (u - big) / each;
    };
    first = owner(group * tiles), count = owner(group * tiles + tiles - 1) - first + 1;
  }
  const int64_t mine = (int64_t)head * a.rows + row, slot = (int64_t)a.group * (2 + D);
  const float* part = a.parts + (first + group) * slot;
  ops_begin();
  ops_next();
  // m and l of all parts, the lane's own last, then their weights
  const int warp = threadIdx.x / 32, split = side / Q, d4 = blockIdx.z * Q + side % Q;
  float top = -INFINITY, sum = 0.f;
  for (uint32_t i = side; i <= count; i += kSide) {
    const float m = __ldcg(i < count ? part + i * slot + at : a.own + mine);
    ls[i][r] = __ldcg(i < count ? part + i * slot + a.group + at : a.own + a.own_rows + mine);
    ms[i][r] = m, top = fmaxf(top, m);
  }
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (split == 0) v = __ldcg(reinterpret_cast<const float4*>(a.own + 2 * a.own_rows + mine * D) + d4);
  // (a warp's threads of a row are eight apart)
  auto of_warp = [&](float x, auto both) {
    x = both(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return both(x, __shfl_xor_sync(0xffffffffu, x, 16));
  };
  auto larger = [](float x, float y) { return fmaxf(x, y); };
  auto plus = [](float x, float y) { return x + y; };
  top = of_warp(top, larger);
  tops[warp][r] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; w++) top = fmaxf(top, tops[w][r]);
  const float ref = top == -INFINITY ? 0.f : top;
  for (uint32_t i = side; i <= count; i += kSide) {
    const float f = exp2a(ms[i][r] - ref);
    ms[i][r] = f, sum += ls[i][r] * f;
  }
  sum = of_warp(sum, plus);
  sums[warp][r] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; w++) sum += sums[w][r];
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
  const int b = row / a.share, c = row - b * a.share, h = head * a.share + c;
  if (a.lse && side == 0 && blockIdx.z == 0) {
    constexpr float kLn2 = 0.6931471805599453f, kLifted = std::is_same_v<T, __half> ? 15.f : 0.f;
    a.lse[b * a.sl_b + h] = (top + (log2f(sum) - kLifted)) * kLn2;
  }
  if (split == 0) {
    const float f = ms[count][r];
    v.x *= f, v.y *= f, v.z *= f, v.w *= f;
  }
#pragma unroll 8
  for (uint32_t i = split; i < count; i += kSplit) {
    const float4 w = __ldcg(reinterpret_cast<const float4*>(part + i * slot + 2 * a.group) + (int64_t)d4 * a.group + at);
    const float f = ms[i][r];
    v.x += w.x * f, v.y += w.y * f, v.z += w.z * f, v.w += w.w * f;
  }
  if (kSplit > 1) {
    const int place = side % Q * kJoinRows + r;
    if (split) more[split][place] = v;
    __syncthreads();
    if (split) return;
#pragma unroll
    for (int i = 1; i < kSplit; i++) {
      const float4 w = more[i][place];
      v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
  }
  const uint32_t w0 = pack2<T>(v.x * inv, v.y * inv), w1 = pack2<T>(v.z * inv, v.w * inv);
  T* out = reinterpret_cast<T*>(a.o) + b * a.so_b + h * a.so_h + d4 * 4;
  if (a.o_even) {
    reinterpret_cast<uint32_t*>(out)[0] = w0, reinterpret_cast<uint32_t*>(out)[1] = w1;
  } else {
    uint16_t* one = reinterpret_cast<uint16_t*>(out);
    one[0] = (uint16_t)w0, one[1] = (uint16_t)(w0 >> 16), one[2] = (uint16_t)w1, one[3] = (uint16_t)(w1 >> 16);
  }
}
template <typename T, int D>
cudaError_t join_by(const Join& a, cudaStream_t st) {
  // With four of the wide CTAs to a multiprocessor what each finds out by itself counts most
  // (128 lanes with 64 heads behind 32767 186 us, 193 with the narrow ones), with fewer the chain of
  // loads (64 lanes with 32 heads behind 8192 43.4 us, 45.3 with the wide ones; 32 lanes with 8 heads to
  // one key-value head behind 32768 26, 42 where one thread adds up all parts of a row's four elements).
  constexpr int kWide = D / 4 < 32 ? D / 4 : 32;
  const dim3 grid((a.rows + kJoinRows - 1) / kJoinRows, a.hkv, D / 4 / kWide);
  if ((int64_t)grid.x * grid.y * grid.z >= 4 * ops_sm_count())
    return ops_launch(join_kernel<T, D, kWide>, grid, kJoinThreads, 0, 0, st, a);
  return ops_launch(join_kernel<T, D, 8>, dim3(grid.x, grid.y, D / 32), kJoinThreads, 0, 0, st, a);
}
template <typename T>
cudaError_t join(const Join& a, int d, cudaStream_t st) {
  return d == 64 ? join_by<T, 64>(a, st) : d == 128 ? join_by<T, 128>(a, st) : join_by<T, 256>(a, st);
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
  if ((int64_t)lanes * q_heads > INT32_MAX || kv_heads > 65535)
    return api_fail(WFST_ERR_INVALID_ARG, "prefix_size: too many heads");
  int64_t own;
  if (const int rc = wfst_attend_size(&own)) return rc;
  const int64_t rows = (int64_t)lanes * (q_heads / kv_heads), group = rows_of_group(rows, head_dim);
  const int64_t groups = (rows + group - 1) / group * kv_heads;
  *bytes = own + ((kMostGrid + groups) * group + (rows * kv_heads + 3) / 4 * 4) * (2 + head_dim) * 4;
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
  const int keys = r->head_dim == 256 ? kKeys<256, 1> : rows == kRows ? kKeys<128, 1> : kKeys<128, 2>;
  const int64_t units = (room + keys - 1) / keys * groups * r->kv_heads;
  if (units > INT32_MAX) return api_fail(WFST_ERR_INVALID_ARG, "attend_prefix: lanes * heads * tokens is too large");
  int64_t own;
  if (const int rc = wfst_attend_size(&own)) return rc;
  OpsDevice guard(dev);
  if (guard.err != cudaSuccess) return api_cuda_fail(guard.err, "attend_prefix: device");
  Join j = {};
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
    if (a.scale2 < FLT_MIN) a.scale2 = FLT_MIN;  // (what is not seen, at -inf, stays there)
    int64_t grid = ops_sm_count();
    if (grid > kMostGrid) grid = kMostGrid;
    if (grid > units) grid = units;
    // Boxes of as many keys as pages hold whole ones of, up to a warp's share of a tile; rows
    // of eight at least, in which the 16-byte pieces are exchanged.
    CUtensorMap maps[2] = {};
    a.box = keys / 4;
    while (a.box > 1 && r->page_size % a.box) a.box /= 2;
    const auto type = r->dtype == WFST_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (a.box < 8 || !map_pool(maps, type, a.kc, r->head_dim, a, ck_s, ck_h, ck_p) ||
        !map_pool(maps + 1, type, a.vc, r->head_dim, a, cv_s, cv_h, cv_p))
      a.box = 0;
    const cudaError_t e = r->dtype == WFST_F16
                              ? by_width<__half>(a, maps, r->head_dim, rows, (int)grid, (cudaStream_t)stream)
                              : by_width<__nv_bfloat16>(a, maps, r->head_dim, rows, (int)grid, (cudaStream_t)stream);
    if (e != cudaSuccess) return api_cuda_fail(e, "attend_prefix launch");
    j.parts = a.parts, j.length = r->prefix_length, j.room = room, j.keys = keys, j.group = rows, j.groups = (int)groups;
    j.grid = (int)grid;
    j.own = a.parts + (kMostGrid + groups * r->kv_heads) * rows * (2 + r->head_dim);
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
  if (const int rc = attend_behind(&b, const_cast<float*>(j.own), stream)) return rc;
  if (!units) return WFST_OK;
  j.o = r->o, j.lse = r->lse;
  j.so_b = stride(r->o_stride[0], r->lanes), j.so_h = stride(r->o_stride[1], r->q_heads), j.sl_b = r->lse_stride;
  j.own_rows = ((int64_t)r->lanes * r->q_heads + 3) / 4 * 4, j.hkv = r->kv_heads, j.share = share, j.rows = r->lanes * share;
  j.o_even = aligned(r->o, 4) && j.so_b % 2 == 0 && j.so_h % 2 == 0;
  const cudaError_t e = r->dtype == WFST_F16 ? join<__half>(j, r->head_dim, (cudaStream_t)stream)
                                             : join<__nv_bfloat16>(j, r->head_dim, (cudaStream_t)stream);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "attend_prefix join launch");
}
