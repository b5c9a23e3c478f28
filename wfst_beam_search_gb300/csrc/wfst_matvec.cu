// wfst_matvec.cu — products with 4-bit weights.
//
//   y[r, n] = bias[n] + sum_k x[r, k] * s[n, k / G] * (c[n, k] - z[n, k / G])
//
// c are codes 0..15, G the group size, z = 8 where no zero points are given.
// A pass has to read the codes (N*K/2 bytes) and the scales; x and y are small
// beside them.  HBM would bound it up to some tens of rows; what it costs to
// bring the codes into the type is the bound that is met before that.  So a code
// is not converted but put in place: as the upper four bits of a mantissa it
// makes the 16-bit number 1 + c / 16, one shift and one logical operation for
// two codes.  A group's sums are in fp32, scaled and added up in fp32, so nothing
// is rounded before y.  Two kernels, by the number of rows:
//   - Few rows: mma.sync fed from registers, eight warps sharing k.  1 x 4096 x
//     4096 takes 4.5 us, 8 x 131072 x 4096 77 us (3.6 TB/s; the floor is 41).
//   - Many rows: tcgen05, the weights widened once into tensor memory by one
//     thread per output, x from shared memory.  64 x 32768 x 4096 takes 40 us,
//     64 x 65536 x 8192 146 us (1.9 TB/s), 64 x 5000 x 1056 in groups of 32 9 us.
// The first one's work goes with the rows, the second one's hardly does, but it
// starts and ends more slowly (barriers, tensor memory, a cluster's sum): 16 x
// 4096 x 4096 is 6.0 against 8.4 us, 32 x 16384 x 4096 31 against 21.  Up to 16
// rows the first one is taken, and above where its CTAs fit on the device at
// once: 64 x 1024 x 4096 is 5.8 against 7.1 us, 32 x 4096 x 4096, which does not
// fit, 10.8 against 9.1, 24 x 5000 x 1056 7.0 against 6.1.
//
// Layout ("packed", made once by wfst_quant_pack): tiles of 128 outputs, in them
// blocks of 64 k, in them eight parts of 16 outputs with 512 bytes each: 16 bytes
// for (t, g), t = 0..3, g = 0..7, hold the codes of outputs g and g + 8 for k = 8 t
// .. 8 t + 7 of either half of the block, a word each (first half g, g + 8, second
// half g, g + 8).  A warp of the one kernel reads 512 consecutive bytes with that,
// a thread of the other one four times 16 bytes without bank conflicts.
#include <cooperative_groups.h>

#include <type_traits>

#include <cuda.h>

#include "wfst_ops.h"

namespace cg = cooperative_groups;

namespace wfst {
namespace {

constexpr int kM = 128;       // outputs of a tile, one to a thread of the first four warps
constexpr int kThreads = kM + 64;
constexpr int kBlock = 64;    // k of a stage
constexpr int kCodes = kM * kBlock / 2;  // bytes of a stage's codes
constexpr int kMaxCluster = 8;
constexpr uint32_t kNap = 20000, kSpins = 1u << 16;  // a wait sleeps so many ns at a time, and gives up after so many times

// Where a code lies in a 16-bit number, and the bits of 1 around it.
template <typename T>
constexpr int kCodeAt = std::is_same_v<T, __half> ? 6 : 3;
template <typename T>
constexpr uint32_t kOnes = std::is_same_v<T, __half> ? 0x3c003c00u : 0x3f803f80u;

// Pair j of a word (k = 2 j and 2 j + 1 of the word's eight) lies where a
// rotation by 4 j to the right brings its two codes to the upper mantissa bits
// of the word's two halves: bits 3-6 and 19-22 for bf16, 6-9 and 22-25 for fp16.
template <int AT>
__global__ void pack_codes(const uint8_t* __restrict__ codes, int64_t n, int64_t k, int64_t blocks, int64_t words,
                           uint32_t* __restrict__ out) {
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += step) {
    const int hi = (int)(i & 1), half = (int)(i >> 1 & 1), g = (int)(i >> 2 & 7), t = (int)(i >> 5 & 3), part = (int)(i >> 7 & 7);
    const int64_t blk = (i >> 10) % blocks, tile = (i >> 10) / blocks;
    const int64_t row = tile * kM + part * 16 + hi * 8 + g, k0 = blk * kBlock + half * 32 + t * 8;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      uint32_t byte = 0;  // past the matrix's edge x or the scale is zero
      if (row < n && k0 + 2 * j < k) byte = codes[row * (k / 2) + k0 / 2 + j];
      const uint32_t pair = (byte & 15u) << AT | (byte >> 4) << (AT + 16);
      w |= __funnelshift_l(pair, pair, 4 * j);
    }
    out[i] = w;
  }
}

// Scales of a tile and group: for each part of 16 outputs and g = 0..7 {s[g],
// s[g + 8]}, with zero points {s[g], s[g + 8], z[g], z[g + 8]}; zero scales past
// the edge.
__global__ void pack_scales(const uint16_t* __restrict__ scales, const uint16_t* __restrict__ zeros, int64_t n,
                            int64_t groups, int64_t groups_p, int64_t count, uint16_t* __restrict__ out) {
  const int per = zeros ? 4 : 2;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < count; i += step) {
    const int j = (int)(i % per), g = (int)(i / per % 8), part = (int)(i / (per * 8) % 8);
    const int64_t grp = i / (per * 64) % groups_p, row = i / (per * 64) / groups_p * kM + part * 16 + (j & 1) * 8 + g;
    uint16_t v = 0;
    if (row < n && grp < groups) v = (j < 2 ? scales : zeros)[row * groups + grp];
    out[i] = v;
  }
}

struct Args {
  const unsigned char* codes;
  const unsigned char* scales;
  const void* x;
  const void* bias;
  void* y;
  int64_t sx, sy;
  int32_t n, k, rows, tiles, blocks, groups_p, group_log;
};

// ---- instructions

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
__device__ __forceinline__ void copy_bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool elected() {
  uint32_t is;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(is));
  return is != 0;
}
// d (+)= a * b; a in tensor memory
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// 32 columns of this warp's 32 lanes from registers
__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}

// 8 columns with one value
__device__ __forceinline__ void tmem_fill8(uint32_t at, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%1,%1,%1,%1,%1,%1,%1};" ::"r"(at), "r"(v) : "memory");
}

// Pair j of a word as 1 + c / 16 of its two codes.
template <typename T>
__device__ __forceinline__ uint32_t widen2(uint32_t w, int j) {
  return ((j ? __funnelshift_r(w, w, 4 * j) : w) & (0x000f000fu << kCodeAt<T>)) | kOnes<T>;
}
template <typename T>
constexpr uint32_t kHalves = std::is_same_v<T, __half> ? 0x3e003e00u : 0x3fc03fc0u;  // 1.5, twice
template <typename T>
__device__ __forceinline__ uint32_t less2(uint32_t v, uint32_t off) {
  using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
  const T2 r = __hsub2(*reinterpret_cast<const T2*>(&v), *reinterpret_cast<const T2*>(&off));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// ---- many rows
//
// A CTA takes 128 outputs, and 128 of its threads one each.  Such a thread stores
// its output's codes to tensor memory as its row of A; x is B; a group's sums are
// read back and scaled by the same thread.  A fifth warp copies ahead, a sixth
// one issues the products; they meet through mbarriers, every wait with a limit.
// The 1 + z / 16 too much is taken off by the tensor cores, which have time: a
// second product of the same x with -(1 + z / 16) in every column of A goes into
// the same fp32 sum, whose terms are then about five times those of sum x (c - z)
// / 16 (at 64 rows 6% faster than subtracting).  Groups of 32 leave no room for it
// in tensor memory, and up to 32 rows it is no faster (24 x 9262 x 7936 24 against
// 23 us): there the threads subtract, exactly.  Both hold for whole z; what z has
// beside its whole part is added as s * rest * sum x (64 x 32768 x 4096 with such z
// 72 us, with whole ones 46).  What bounds it is the chain of a stage (wait, widen,
// store, product, read back) and the instructions in it, not HBM.  A non-finite x
// can make NaN of a sum that would be infinite, in its own row of y only.
//
// Sizes that go with N rows of x (32 or 64) and groups of 32 (SUB):

// whether the tensor cores take off 1 + z / 16
template <int N, bool SUB>
constexpr bool kFold = !SUB && N != 32;
// tensor memory: two stages of A (32 columns each); two constants for kFold (8);
// two sums of N columns (four with SUB)
template <int N, bool SUB>
constexpr int kSumAt = 64 + (kFold<N, SUB> ? 16 : 0);
template <int N, bool SUB>
constexpr int kUsed = kSumAt<N, SUB> + (SUB ? 4 : 2) * N;
template <int N, bool SUB>
constexpr int kColumns = kUsed<N, SUB> <= 128 ? 128 : kUsed<N, SUB> <= 256 ? 256 : 512;
template <int N>
constexpr int kStages = N == 64 ? 7 : 6;
template <int N, bool SUB, bool ZERO>
constexpr int kSlot = (N * 128 + kCodes + (SUB ? 2 : 1) * kM * (ZERO ? 4 : 2) + 1023) / 1024 * 1024;
// CTAs of a multiprocessor: two if its 512 columns hold them, and no more, since
// one that waits for columns would hold up its cluster, and three only share what
// two get done (32 x 8192 x 4096 12 us, with three, split in more shares, 16);
// shared memory sees to it
template <int N, bool SUB>
constexpr int kResident = kColumns<N, SUB> <= 256 ? 2 : 1;
template <int N, bool SUB, bool ZERO>
constexpr int kSmem = 1024 + (kStages<N> * kSlot<N, SUB, ZERO> > 233472 / (kResident<N, SUB> + 1)
                                  ? kStages<N> * kSlot<N, SUB, ZERO>
                                  : 233472 / (kResident<N, SUB> + 1));

// One CTA: 128 outputs by N rows of x, a share of k; a cluster adds up its
// CTAs' shares in order.  SUB: groups of 32, two to a stage; otherwise a group
// is whole stages.
template <typename T, int N, bool SUB, bool ZERO>
__global__ void __launch_bounds__(kThreads, kResident<N, SUB>)
    matvec_wide(const Args a, const __grid_constant__ CUtensorMap x_map) {
  extern __shared__ unsigned char raw_smem[];
  constexpr int S = kStages<N>, kSize = kSlot<N, SUB, ZERO>, kParts = SUB ? 2 : 1, kScale = ZERO ? 4 : 2;
  constexpr bool FOLD = kFold<N, SUB>;
  // a slot is filled, a slot is free; A is written, the products of a stage are through
  __shared__ __align__(8) uint64_t bars[2 * S + 4];
  __shared__ uint32_t tmem_at;
  __shared__ int failed;
  __shared__ __align__(16) float sums[ZERO ? 4 : 1][kParts][ZERO ? N : 4];  // of x's rows, a copy for each warp
  cg::cluster_group cl = cg::this_cluster();
  const int shares = (int)cl.num_blocks(), share = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tile = blockIdx.x / shares, row0 = blockIdx.y * N;
  const int b0 = (int)((int64_t)a.blocks * share / shares), count = (int)((int64_t)a.blocks * (share + 1) / shares) - b0;
  // x's tiles are read by the tensor cores in a pattern of 1024 bytes
  unsigned char* ring = raw_smem + ((1024 - ((uint32_t)__cvta_generic_to_shared(raw_smem) & 1023)) & 1023);
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  const uint32_t bar = (uint32_t)__cvta_generic_to_shared(bars);
  auto filled = [&](int slot) { return bar + slot * 8; };
  auto is_free = [&](int slot) { return bar + (S + slot) * 8; };
  auto a_in = [&](int p) { return bar + (2 * S + p) * 8; };
  auto through = [&](int p) { return bar + (2 * S + 2 + p) * 8; };

  if (tid == 0) {
    failed = 0;
    for (int i = 0; i < 2 * S + 4; i++) {
      const int n = i < S || i >= 2 * S + 2 ? 1 : 4;
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar + i * 8), "r"(n) : "memory");
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  ops_begin();
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(&tmem_at)),
                 "n"(kColumns<N, SUB>)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_at;
  ops_next();
  bool good = true;

  float acc[N];
  if (warp == 4) {
    // ---- copies: x (rows of 128 bytes, 16-byte pieces exchanged by row), codes and scales
    int slot = 0, round = 0, issued = 0;  // issued: by the elected lane, the others have none
    for (int i = 0; i < count; i++) {
      const int blk = b0 + i;
      if (round) good = good && wait_bar(is_free(slot), (round - 1) & 1);
      if (elected() && good) {
        issued = i + 1;
        const uint32_t dst = ring_at + slot * kSize;
        constexpr uint32_t bytes = N * 128 + kCodes + kParts * kM * kScale;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(filled(slot)), "n"(bytes) : "memory");
        const int grp = SUB ? blk * 2 : blk * kBlock >> a.group_log;
        copy_bulk(dst + N * 128, a.codes + ((int64_t)tile * a.blocks + blk) * kCodes, kCodes, filled(slot));
        copy_bulk(dst + N * 128 + kCodes, a.scales + ((int64_t)tile * a.groups_p + grp) * (kM * kScale),
                  kParts * kM * kScale, filled(slot));
        // (zeros come for rows and k past x's ends)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(&x_map), "r"(blk * kBlock), "r"(row0), "r"(filled(slot))
            : "memory");
      }
      __syncwarp();
      if (++slot == S) slot = 0, round++;
    }
    // nothing may be on its way when the CTA ends, nor where a wait gave up
    for (int i = issued > S ? issued - S : 0; i < issued; i++) good = wait_bar(filled(i % S), (i / S) & 1) && good;
    __syncwarp();
  } else if (warp == 5) {
    // ---- products.  kind::f16: fp32 sums, both operands T with k innermost, N columns, 128 rows
    constexpr uint32_t kType = std::is_same_v<T, __half> ? 0u : 1u;
    constexpr uint32_t idesc = 1u << 4 | kType << 7 | kType << 10 | (uint32_t)(N / 8) << 17 | (uint32_t)(kM / 16) << 24;
    // x: rows of 128 bytes, groups of eight rows 1024 bytes apart, pieces exchanged within 128 bytes
    const uint64_t desc0 = (uint64_t)(ring_at >> 4 & 0x3fffu) | 1ull << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
    int sum = 0, slot = 0, phase = 0, issued = 0;  // issued: as above
    bool begins = true;
    for (int i = 0; i < count; i++) {
      const int p = i & 1, blk = b0 + i;
      good = good && wait_bar(filled(slot), phase) && wait_bar(a_in(p), (i / 2) & 1);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint64_t desc = desc0 + (uint64_t)(slot * (kSize >> 4));
      if (elected() && good) {
        issued = i + 1;
        const uint32_t d = tmem + kSumAt<N, SUB> + sum * kParts * N;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          product(d + (SUB ? j / 2 * N : 0), tmem + p * 32 + j * 8, desc + 2 * j, idesc, SUB ? j % 2 != 0 : j || !begins);
          if (FOLD) product(d, tmem + 64 + (ZERO ? sum * 8 : 0), desc + 2 * j, idesc, true);
        }
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(through(p)) : "memory");
      }
      __syncwarp();
      begins = SUB || ((blk + 1) * kBlock & ((1 << a.group_log) - 1)) == 0;
      if (begins) sum ^= 1;
      if (++slot == S) slot = 0, phase ^= 1;
    }
    // nor a product when its tensor memory is given back
    for (int i = issued > 2 ? issued - 2 : 0; i < issued; i++) good = wait_bar(through(i & 1), (i / 2) & 1) && good;
    __syncwarp();
  } else {
    // ---- codes into the operand type; the groups' sums, scaled
    const uint32_t mine = tmem + (uint32_t)(warp * 32 << 16);  // this warp's lanes
#pragma unroll
    for (int i = 0; i < N; i++) acc[i] = 0.f;
    auto add_up = [&](int column, float scale) {
#pragma unroll
      for (int i = 0; i < N; i += 16) {
        uint32_t r[16];
        tmem_load16(r, mine + column + i);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int j = 0; j < 16; j++) acc[i + j] += scale * __uint_as_float(r[j]);
      }
    };
    if (FOLD && !ZERO) tmem_fill8(mine + 64, pack2<T>(-1.5f, -1.5f));
    int slot = 0, phase = 0, sum = 0, old = 0;
    bool begins = true;
    // of the two stages before: where a group ended, and its scale
    int end0 = -1, end1 = -1;
    float scale0[kParts], scale1[kParts];
    auto step = [&](int i, int& end, float (&scale)[kParts]) {
      const int p = i & 1;
      if (i >= 2) {  // the products of the stage before the last one are through: its slot and A are free
        good = good && wait_bar(through(p), (i / 2 - 1) & 1);
        if (lane == 0) arrive(is_free(old));
        if (++old == S) old = 0;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (end >= 0) {
#pragma unroll
          for (int h = 0; h < kParts; h++) add_up(kSumAt<N, SUB> + (end * kParts + h) * N, scale[h]);
        }
      }
      end = -1;
      if (i >= count) return;
      good = good && wait_bar(filled(slot), phase);
      const unsigned char* stage = ring + slot * kSize;
      float s_one[kParts], rest[kParts];
      uint32_t one[kParts];
#pragma unroll
      for (int h = 0; h < kParts; h++) {
        // {s[g], s[g + 8]} or {s[g], s[g + 8], z[g], z[g + 8]}
        const T* at = reinterpret_cast<const T*>(stage + N * 128 + kCodes + h * kM * kScale) +
                      (tid / 16 * 8 + tid % 8) * kScale + tid / 8 % 2;
        s_one[h] = to_f32(at[0]);
        rest[h] = 0.f;
        one[h] = pack2<T>(1.5f, 1.5f);
        if (ZERO) {
          const float z = to_f32(at[2]), whole = fminf(fmaxf(rintf(z), 0.f), 15.f);
          rest[h] = whole - z;
          one[h] = pack2<T>(1.f + whole * 0.0625f, 1.f + whole * 0.0625f);
        }
        scale[h] = 16.f * s_one[h];
      }
      const uint4* words = reinterpret_cast<const uint4*>(stage + N * 128 + tid / 16 * 512) + tid % 8;
      const bool upper = tid / 8 % 2;
      uint32_t w[8];
#pragma unroll
      for (int t = 0; t < 4; t++) {
        const uint4 v = words[t * 8];
        w[t] = upper ? v.y : v.x;
        w[4 + t] = upper ? v.w : v.z;
      }
      uint32_t r[32];
#pragma unroll
      for (int j = 0; j < 32; j++) {
        r[j] = widen2<T>(w[j / 4], j % 4);
        if (!FOLD) r[j] = less2<T>(r[j], one[SUB ? j / 16 : 0]);
      }
      tmem_store32(mine + p * 32, r);
      if (FOLD && ZERO && begins) tmem_fill8(mine + 64 + sum * 8, one[0] ^ 0x80008000u);
      if (ZERO) {  // zero points that are not whole
        bool some = false;
#pragma unroll
        for (int h = 0; h < kParts; h++) some = some || !(rest[h] == 0.f);
        if (__any_sync(0xffffffffu, some)) {  // each warp sums the rows of x, a lane one or two
          __syncwarp();
#pragma unroll
          for (int j = lane; j < N; j += 32) {
            float t[kParts] = {};
#pragma unroll
            for (int c = 0; c < 8; c++) {
              const uint4 v = *reinterpret_cast<const uint4*>(stage + j * 128 + ((c ^ (j & 7)) * 16));
              const float2 f0 = unpack2<T>(v.x), f1 = unpack2<T>(v.y), f2 = unpack2<T>(v.z), f3 = unpack2<T>(v.w);
              t[SUB ? c / 4 : 0] += ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
            }
#pragma unroll
            for (int h = 0; h < kParts; h++) sums[warp][h][j] = t[h];
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < N; j += 4)
#pragma unroll
            for (int h = 0; h < kParts; h++) {
              const float4 t = *reinterpret_cast<const float4*>(&sums[warp][h][j]);
              const float f = s_one[h] * rest[h];
              acc[j] += f * t.x, acc[j + 1] += f * t.y, acc[j + 2] += f * t.z, acc[j + 3] += f * t.w;
            }
        }
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(a_in(p));
      if (++slot == S) slot = 0, phase ^= 1;
      begins = SUB || ((b0 + i + 1) * kBlock & ((1 << a.group_log) - 1)) == 0;
      if (begins || i + 1 == count) end = sum;
      if (begins) sum ^= 1;
    };
    for (int i = 0; i < count + 2; i += 2) {
      step(i, end0, scale0);
      if (i + 1 < count + 2) step(i + 1, end1, scale1);
    }
  }
  if (!good) failed = 1;
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  // (before the cluster meets: a CTA elsewhere may be waiting for the columns)
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kColumns<N, SUB>));
  if (warp < 4 && failed) {  // a wait gave up: the result says so
#pragma unroll
    for (int i = 0; i < N; i++) acc[i] = __int_as_float(0x7fffffff);
  }

  auto write = [&](int r, int n, float v) {
    if (row0 + r >= a.rows || n >= a.n) return;
    if (a.bias) v += to_f32(reinterpret_cast<const T*>(a.bias)[n]);
    reinterpret_cast<T*>(a.y)[(row0 + r) * a.sy + n] = from_f32<T>(v);
  };
  if (shares == 1) {
    if (warp < 4) {
#pragma unroll
      for (int i = 0; i < N; i++) write(i, tile * kM + tid, acc[i]);
    }
    return;
  }
  float* part = reinterpret_cast<float*>(ring);  // [row of x][output]
  if (warp < 4) {
#pragma unroll
    for (int i = 0; i < N; i++) part[i * kM + tid] = acc[i];
  }
  cl.sync();
  if (warp < 4) {
    // a warp takes a row at a time, a lane four of its outputs
    for (int i = share + warp * shares; i < N && row0 + i < a.rows; i += 4 * shares) {
      float4 v[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; r++)
        v[r] = r < shares ? *cl.map_shared_rank(reinterpret_cast<float4*>(part + i * kM) + lane, r) : make_float4(0.f, 0.f, 0.f, 0.f);
      float4 all = v[0];
#pragma unroll
      for (int r = 1; r < kMaxCluster; r++) all.x += v[r].x, all.y += v[r].y, all.z += v[r].z, all.w += v[r].w;
      const float w[4] = {all.x, all.y, all.z, all.w};
#pragma unroll
      for (int j = 0; j < 4; j++) write(i, tile * kM + lane * 4 + j, w[j]);
    }
  }
  cl.sync();  // no CTA leaves while another may read its shared memory
}

// x as the tensor cores' copies want it: boxes of N rows by 64 k
CUresult map_x(CUtensorMap* map, const Args& a, CUtensorMapDataType type, int n) {
  static const auto encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult how;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &how) != cudaSuccess)
      fn = nullptr;
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(fn);
  }();
  if (!encode) return CUDA_ERROR_NOT_SUPPORTED;
  const cuuint64_t size[2] = {(cuuint64_t)a.k, (cuuint64_t)a.rows}, stride[1] = {(cuuint64_t)a.sx * 2};
  const cuuint32_t box[2] = {kBlock, (cuuint32_t)n}, step[2] = {1, 1};
  return encode(map, type, 2, const_cast<void*>(a.x), size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <typename T, int N, bool SUB, bool ZERO>
cudaError_t launch_wide(const Args& a, cudaStream_t st) {
  auto* fn = matvec_wide<T, N, SUB, ZERO>;
  constexpr int smem = kSmem<N, SUB, ZERO>;
  static OpsOnce once;
  if (const int dev = ops_current(); !once(dev)) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    once.set(dev);
  }
  CUtensorMap map;
  if (map_x(&map, a, std::is_same_v<T, __half> ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, N) !=
      CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  // k is shared among as many CTAs as cost least: rounds of CTAs times the stages
  // of one, its start and end taking about as long as kEnds stages (64 x 5000 x
  // 1056 9 us, without it, split as far as CTAs fit, 15; 64 x 32768 x 4096 41, 50)
  constexpr int kEnds = 7;
  const int rows = (a.rows + N - 1) / N;
  const int64_t slots = (int64_t)ops_sm_count() * kResident<N, SUB>, ctas = (int64_t)a.tiles * rows;
  int shares = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= kMaxCluster && s <= a.blocks; s++) {
    const int64_t cost = (ctas * s + slots - 1) / slots * ((a.blocks + s - 1) / s + kEnds);
    if (cost < least) least = cost, shares = s;
  }
  return ops_launch(fn, dim3((unsigned)a.tiles * shares, rows), kThreads, smem, shares, st, a, map);
}

template <typename T, int N>
cudaError_t wide(const Args& a, bool zeros, cudaStream_t st) {
  if (a.group_log == 5) return zeros ? launch_wide<T, N, true, true>(a, st) : launch_wide<T, N, true, false>(a, st);
  return zeros ? launch_wide<T, N, false, true>(a, st) : launch_wide<T, N, false, false>(a, st);
}

// ---- few rows

constexpr int kWarps = 8;
// CTAs of a multiprocessor that the registers are held down for: 8 x 32768 x 4096
// in groups of 32 with zero points 28 us; at three the registers spill, 39
constexpr int kHeld = 2;

__device__ __forceinline__ uint32_t first_of(uint32_t v) { return v; }
__device__ __forceinline__ uint32_t first_of(uint2 v) { return v.x; }
__device__ __forceinline__ uint32_t second_of(uint32_t) { return 0; }
__device__ __forceinline__ uint32_t second_of(uint2 v) { return v.y; }

// One CTA: MT parts of 16 outputs by NT*8 rows; its warps share the blocks of k
// among them (warp w takes blocks w, w + kWarps, ...) and add up at the end, in
// warp order.  A warp loads the codes and scales of U blocks while it works on the
// U before.  (Copies into a ring in shared memory, and CTAs that stay and load
// across the parts' ends, took 10 to 20% longer: the instructions count.)  K is
// permuted within the instructions' steps, alike on both sides: lane (g, t) has k
// = 8 t .. 8 t + 7 of a half block, of outputs g and g + 8 and of row g of x.
// SUB: groups of 32, two to a block; otherwise a group is whole blocks.
template <typename T, int MT, int NT, int U, bool SUB, bool ZERO>
__global__ void __launch_bounds__(kWarps * 32, kHeld) matvec_narrow(const Args a) {
  extern __shared__ float red[];  // [warp][row of x][kOut]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  ops_begin();
  const int part0 = blockIdx.x * MT, row0 = blockIdx.y * (NT * 8), parts = (a.n + 15) / 16;
  constexpr int kParts = SUB ? 2 : 1;      // scale groups of a block
  constexpr int kSteps = 4 / kParts;       // matrix steps of a group
  constexpr int kOut = MT * 16;
  using Scale = std::conditional_t<ZERO, uint2, uint32_t>;  // scales (and zero points) of outputs g, g + 8
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int i = 0; i < 4; i++) acc[m][j][i] = 0.f;

  // rows of x past the last one read the last one; their results are dropped
  const T* xp[NT];
#pragma unroll
  for (int j = 0; j < NT; j++)
    xp[j] = reinterpret_cast<const T*>(a.x) + (int64_t)min(row0 + j * 8 + g, a.rows - 1) * a.sx + t * 8;
  const uint4* cp[MT];
  const Scale* sp[MT];
#pragma unroll
  for (int m = 0; m < MT; m++) {
    const int part = min(part0 + m, parts - 1);  // one past the end repeats the last one
    cp[m] = reinterpret_cast<const uint4*>(a.codes) + ((int64_t)(part / 8) * a.blocks * 8 + part % 8) * 32 + t * 8 + g;
    sp[m] = reinterpret_cast<const Scale*>(a.scales) + ((int64_t)(part / 8) * a.groups_p * 8 + part % 8) * 8 + g;
  }

  uint4 next[U][MT];
  Scale next_s[U][MT][kParts];
  auto load = [&](int b0) {
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int blk = b0 + u * kWarps;
      if (blk < a.blocks) {
#pragma unroll
        for (int m = 0; m < MT; m++) {
          next[u][m] = ops_load_once(cp[m] + (int64_t)blk * 256);
#pragma unroll
          for (int p = 0; p < kParts; p++)
            next_s[u][m][p] = ops_load(sp[m] + (int64_t)(SUB ? blk * 2 + p : blk * kBlock >> a.group_log) * 64);
        }
      }
    }
  };
  load(warp);
  for (int b0 = warp; b0 < a.blocks; b0 += U * kWarps) {
    uint4 c[U][MT];
    Scale cs[U][MT][kParts];
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int m = 0; m < MT; m++) {
        c[u][m] = next[u][m];
#pragma unroll
        for (int p = 0; p < kParts; p++) cs[u][m][p] = next_s[u][m][p];
      }
    load(b0 + U * kWarps);
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int blk = b0 + u * kWarps;
      if (blk >= a.blocks) break;
      uint4 xv[NT][2];
      const bool second = blk * kBlock + 32 < a.k;  // k is whole halves of a block
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const uint4* p = reinterpret_cast<const uint4*>(xp[j] + blk * kBlock);
        xv[j][0] = ops_load(p);
        xv[j][1] = second ? ops_load(p + 4) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int p = 0; p < kParts; p++) {
        float2 sc[MT], off[MT];  // 16 s and (8 - z) s of outputs g and g + 8
#pragma unroll
        for (int m = 0; m < MT; m++) {
          sc[m] = unpack2<T>(first_of(cs[u][m][p]));
          if (ZERO) {
            const float2 z = unpack2<T>(second_of(cs[u][m][p]));
            off[m] = make_float2(sc[m].x * (8.f - z.x), sc[m].y * (8.f - z.y));
          }
          sc[m].x *= 16.f;
          sc[m].y *= 16.f;
        }
        if (ZERO) {
#pragma unroll
          for (int j = 0; j < NT; j++) {
            float sum[4] = {0.f, 0.f, 0.f, 0.f};  // every row is the same: columns 2t, 2t + 1
#pragma unroll
            for (int s = p * kSteps; s < (p + 1) * kSteps; s++) {
              const uint32_t* xw = reinterpret_cast<const uint32_t*>(xv[j]) + 2 * s;
              mma16816<T>(sum, kOnes<T>, kOnes<T>, kOnes<T>, kOnes<T>, xw[0], xw[1]);
            }
#pragma unroll
            for (int m = 0; m < MT; m++) {
              acc[m][j][0] += off[m].x * sum[0];
              acc[m][j][1] += off[m].x * sum[1];
              acc[m][j][2] += off[m].y * sum[0];
              acc[m][j][3] += off[m].y * sum[1];
            }
          }
        }
#pragma unroll
        for (int m = 0; m < MT; m++) {
          float d[NT][4];
#pragma unroll
          for (int j = 0; j < NT; j++) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
#pragma unroll
          for (int s = p * kSteps; s < (p + 1) * kSteps; s++) {
            const uint32_t w0 = s / 2 ? c[u][m].z : c[u][m].x, w8 = s / 2 ? c[u][m].w : c[u][m].y;
            const uint32_t a0 = less2<T>(widen2<T>(w0, s % 2 * 2), kHalves<T>), a1 = less2<T>(widen2<T>(w8, s % 2 * 2), kHalves<T>);
            const uint32_t a2 = less2<T>(widen2<T>(w0, s % 2 * 2 + 1), kHalves<T>),
                           a3 = less2<T>(widen2<T>(w8, s % 2 * 2 + 1), kHalves<T>);
#pragma unroll
            for (int j = 0; j < NT; j++) {
              const uint32_t* xw = reinterpret_cast<const uint32_t*>(xv[j]) + 2 * s;
              mma16816<T>(d[j], a0, a1, a2, a3, xw[0], xw[1]);
            }
          }
#pragma unroll
          for (int j = 0; j < NT; j++) {
            acc[m][j][0] += sc[m].x * d[j][0];
            acc[m][j][1] += sc[m].x * d[j][1];
            acc[m][j][2] += sc[m].y * d[j][2];
            acc[m][j][3] += sc[m].y * d[j][3];
          }
        }
      }
    }
  }

  ops_next();  // (here, not before the loop: 1 x 4096 x 4096 4.5 us, at the start 5.6)
  float* mine = red + warp * (NT * 8 * kOut);
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int i = 0; i < 4; i++) mine[(j * 8 + 2 * t + (i & 1)) * kOut + m * 16 + g + (i >> 1) * 8] = acc[m][j][i];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 8 * kOut; i += kWarps * 32) {
    const int r = row0 + i / kOut, n = part0 * 16 + i % kOut;
    if (r >= a.rows || n >= a.n) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) v += red[w * (NT * 8 * kOut) + i];
    if (a.bias) v += to_f32(reinterpret_cast<const T*>(a.bias)[n]);
    reinterpret_cast<T*>(a.y)[r * a.sy + n] = from_f32<T>(v);
  }
}

template <typename T, int MT, int NT, int U, bool SUB, bool ZERO>
cudaError_t launch_narrow(const Args& a, cudaStream_t st) {
  constexpr int smem = kWarps * NT * 8 * MT * 16 * (int)sizeof(float);
  static_assert(smem <= 48 * 1024);
  const dim3 grid(((a.n + 15) / 16 + MT - 1) / MT, (a.rows + NT * 8 - 1) / (NT * 8));
  return ops_launch(matvec_narrow<T, MT, NT, U, SUB, ZERO>, grid, kWarps * 32, smem, 0, st, a);
}

template <typename T, int MT, int NT, int U>
cudaError_t narrow(const Args& a, bool zeros, cudaStream_t st) {
  if (a.group_log == 5)
    return zeros ? launch_narrow<T, MT, NT, U, true, true>(a, st) : launch_narrow<T, MT, NT, U, true, false>(a, st);
  return zeros ? launch_narrow<T, MT, NT, U, false, true>(a, st) : launch_narrow<T, MT, NT, U, false, false>(a, st);
}

template <typename T>
cudaError_t by_rows(const Args& a, bool zeros, cudaStream_t st) {
  const int64_t parts = ((int64_t)a.n + 15) / 16, room = (int64_t)kHeld * ops_sm_count();
  if (a.rows <= 16 || parts * ((a.rows + 15) / 16) <= room) {
    // two parts of outputs share a CTA's loads of x where that leaves CTAs for
    // every place: 8 x 131072 x 4096 77 us, with one part 81
    const bool two = parts >= 2 * room;
    if (a.rows <= 8) return two ? narrow<T, 2, 1, 2>(a, zeros, st) : narrow<T, 1, 1, 4>(a, zeros, st);
    return two ? narrow<T, 2, 2, 2>(a, zeros, st) : narrow<T, 1, 2, 4>(a, zeros, st);
  }
  if (a.rows <= 32) return wide<T, 32>(a, zeros, st);
  return wide<T, 64>(a, zeros, st);
}

constexpr int32_t kMost = INT32_MAX - 256;  // rounded up to whole tiles they still fit an int

struct Sizes {
  int64_t tiles, blocks, groups, groups_p, code_bytes, bytes;
};

// NULL, or what is wrong with the matrix's sizes.
const char* sizes(int32_t n, int32_t k, int32_t group, bool zeros, Sizes* s) {
  if (n < 1 || k < 1 || n > kMost || k > kMost) return "n and k must be between 1 and 2^31 - 257";
  if (group != 32 && group != 64 && group != 128 && group != 256) return "group must be 32, 64, 128 or 256";
  if (k % group) return "k must be a multiple of group";
  s->tiles = ((int64_t)n + kM - 1) / kM;
  s->blocks = ((int64_t)k + kBlock - 1) / kBlock;
  s->groups = k / group;
  s->groups_p = group == 32 ? s->blocks * 2 : s->groups;
  s->code_bytes = s->tiles * s->blocks * kCodes;
  s->bytes = s->code_bytes + s->tiles * s->groups_p * (kM * (zeros ? 4 : 2));
  return nullptr;
}

}  // namespace

int ops_sm_count() {
  static std::atomic<int> count[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return 152;
  int v = count[dev].load(std::memory_order_relaxed);
  if (!v) {
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    count[dev].store(v = v > 0 ? v : 152, std::memory_order_relaxed);
  }
  return v;
}

}  // namespace wfst

using namespace wfst;

extern "C" int wfst_quant_size(int32_t n, int32_t k, int32_t group, int32_t zeros, int64_t* bytes) {
  Sizes s;
  if (!bytes) return api_fail(WFST_ERR_INVALID_ARG, "quant_size: NULL argument");
  if (const char* why = sizes(n, k, group, zeros != 0, &s)) return api_fail(WFST_ERR_INVALID_ARG, why);
  *bytes = s.bytes;
  return WFST_OK;
}

extern "C" int wfst_quant_pack(const uint8_t* codes, const void* scales, const void* zeros, int32_t dtype, int32_t n,
                               int32_t k, int32_t group, void* packed, void* stream) {
  Sizes s;
  if (!codes || !scales || !packed) return api_fail(WFST_ERR_INVALID_ARG, "quant_pack: NULL argument");
  if (const char* why = sizes(n, k, group, zeros != nullptr, &s)) return api_fail(WFST_ERR_INVALID_ARG, why);
  if (dtype != WFST_F16 && dtype != WFST_BF16) return api_fail(WFST_ERR_INVALID_ARG, "quant_pack: bad dtype");
  if (!aligned(packed, 16)) return api_fail(WFST_ERR_INVALID_ARG, "quant_pack: packed must be 16-byte aligned");
  const int dev = ops_device(-1, {codes, scales, zeros, packed});
  if (dev < 0) return api_fail(WFST_ERR_INVALID_ARG, "quant_pack: every array must be device memory of one device");
  OpsDevice guard(dev);
  if (guard.err != cudaSuccess) return api_cuda_fail(guard.err, "quant_pack: device");
  cudaStream_t st = (cudaStream_t)stream;
  const int grid = ops_sm_count() * 8;
  auto* pack = dtype == WFST_F16 ? pack_codes<kCodeAt<__half>> : pack_codes<kCodeAt<__nv_bfloat16>>;
  pack<<<grid, 256, 0, st>>>(codes, n, k, s.blocks, s.code_bytes / 4, reinterpret_cast<uint32_t*>(packed));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return api_cuda_fail(e, "quant_pack: pack_codes launch");
  pack_scales<<<grid, 256, 0, st>>>(reinterpret_cast<const uint16_t*>(scales), reinterpret_cast<const uint16_t*>(zeros),
                                    n, s.groups, s.groups_p, (s.bytes - s.code_bytes) / 2,
                                    reinterpret_cast<uint16_t*>(static_cast<char*>(packed) + s.code_bytes));
  e = cudaGetLastError();
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "quant_pack: pack_scales launch");
}

extern "C" int wfst_matvec_quant(const wfst_matvec_args* r, void* stream) {
  Sizes s;
  if (!r) return api_fail(WFST_ERR_INVALID_ARG, "matvec_quant: NULL argument");
  if (const char* why = sizes(r->n, r->k, r->group, r->zeros != 0, &s)) return api_fail(WFST_ERR_INVALID_ARG, why);
  if (r->rows < 0) return api_fail(WFST_ERR_INVALID_ARG, "matvec_quant: rows must be >= 0");
  if (r->dtype != WFST_F16 && r->dtype != WFST_BF16) return api_fail(WFST_ERR_INVALID_ARG, "matvec_quant: bad dtype");
  if (r->rows == 0) return WFST_OK;
  if (!r->packed || !r->x || !r->y) return api_fail(WFST_ERR_INVALID_ARG, "matvec_quant: NULL argument");
  if (!aligned(r->packed, 16) || !aligned(r->x, 16) || (r->rows > 1 && r->stride_x % 8))
    return api_fail(WFST_ERR_INVALID_ARG, "matvec_quant: packed and the rows of x must be 16-byte aligned");
  if (r->rows > 1 && (r->stride_x < r->k || r->stride_y < r->n))
    return api_fail(WFST_ERR_INVALID_ARG, "matvec_quant: stride_x must be >= k and stride_y >= n");
  if (r->rows > 65535 * 64) return api_fail(WFST_ERR_INVALID_ARG, "matvec_quant: too many rows");
  const int dev = ops_device(r->device, {r->packed, r->x, r->bias, r->y});
  if (dev < 0) return api_fail(WFST_ERR_INVALID_ARG, "matvec_quant: every array must be device memory of one device");
  OpsDevice guard(dev);
  if (guard.err != cudaSuccess) return api_cuda_fail(guard.err, "matvec_quant: device");
  Args a;
  a.codes = static_cast<const unsigned char*>(r->packed);
  a.scales = a.codes + s.code_bytes;
  a.x = r->x;
  a.bias = r->bias;
  a.y = r->y;
  a.sx = r->rows > 1 ? r->stride_x : 0;
  a.sy = r->rows > 1 ? r->stride_y : 0;
  a.n = r->n;
  a.k = r->k;
  a.rows = r->rows;
  a.tiles = (int32_t)s.tiles;
  a.blocks = (int32_t)s.blocks;
  a.groups_p = (int32_t)s.groups_p;
  a.group_log = 5;
  while (1 << a.group_log < r->group) a.group_log++;
  cudaStream_t st = (cudaStream_t)stream;
  const bool zeros = r->zeros != 0;
  const cudaError_t e =
      r->dtype == WFST_F16 ? by_rows<__half>(a, zeros, st) : by_rows<__nv_bfloat16>(a, zeros, st);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "matvec_quant launch");
}
