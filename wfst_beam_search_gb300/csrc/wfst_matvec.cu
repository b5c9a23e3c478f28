// wfst_matvec.cu — products with 4-bit weights.
//
//   y[r, n] = bias[n] + sum_k x[r, k] * s[n, k / G] * (c[n, k] - z[n, k / G])
//
// c are codes 0..15, G the group size, z = 8 where no zero points are given.
// A pass has to read the codes (N*K/2 bytes) and the scales; x and y are small
// beside them, so HBM bounds it up to some tens of rows.
//
// Matrix instructions do the products (m16n8k16: 16 outputs x 8 rows of x),
// also for one row: products on the general lanes would not keep up with HBM.
// What it costs to bring codes into the instructions' types is the next bound,
// so a code is not converted but put in place: as the upper four bits of a
// mantissa it makes the 16-bit number 1 + c / 16, one shift and one logical
// operation for two codes, and less 1.5 it is (c - 8) / 16, exactly.  A group's
// fp32 sum is scaled once, so nothing is rounded before y.  With zero points the
// group adds s * (8 - z) * sum x, the sum of x coming from the same instruction
// with ones in place of the codes, once for all outputs of a warp.
//
// Layout ("packed", made once by wfst_quant_pack): tiles of 16 outputs, in
// them blocks of 64 k, in them 16 bytes per lane, so that a warp's load is 512
// consecutive bytes.  Inside a block, k is permuted so that a lane's x
// elements are two runs of 8 consecutive ones: lane (g, t) = (lane / 4, lane %
// 4) holds k = 64*blk + 32*(s/2) + 8*t + 4*(s%2) + {0..3} of outputs g and
// g + 8 in word s, and uses them in step s as the instruction's columns 2t,
// 2t+1, 2t+8, 2t+9.  The same permutation on both operands leaves the sum
// unchanged, and steps 0-1 and 2-3 are the block's two halves, as groups of 32
// want it.
#include <type_traits>

#include "wfst_ops.h"

namespace wfst {
namespace {

constexpr int kWarps = 8;

// Pair j of a word (0: output g, k 0/1; 1: output g+8, k 0/1; 2: output g, k
// 2/3; 3: output g+8, k 2/3) lies where a rotation by 4 j to the right brings
// its two codes to the upper mantissa bits of the word's two halves: bits 3-6
// and 19-22 for bf16, bits 6-9 and 22-25 for fp16.
template <int AT>
__global__ void pack_codes(const uint8_t* __restrict__ codes, int64_t n, int64_t k, int64_t blocks, int64_t words,
                           uint32_t* __restrict__ out) {
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += step) {
    const int s = (int)(i & 3), lane = (int)(i >> 2 & 31);
    const int64_t blk = (i >> 7) % blocks, tile = (i >> 7) / blocks;
    const int64_t k0 = blk * 64 + (s >> 1) * 32 + (lane & 3) * 8 + (s & 1) * 4;
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int64_t row = tile * 16 + (lane >> 2) + (j & 1) * 8, kk = k0 + (j >> 1) * 2;
      uint32_t byte = 0;  // past the matrix's edge x or the scale is zero
      if (row < n && kk < k) byte = codes[row * (k / 2) + kk / 2];
      const uint32_t pair = (byte & 15u) << AT | (byte >> 4) << (AT + 16);
      w |= __funnelshift_l(pair, pair, 4 * j);
    }
    out[i] = w;
  }
}

// Scales of a tile and group: for g = 0..7 {s[g], s[g+8]} and, with zero
// points, {z[g], z[g+8]} behind them; zero scales past the edge.
__global__ void pack_scales(const uint16_t* __restrict__ scales, const uint16_t* __restrict__ zeros, int64_t n,
                            int64_t groups, int64_t groups_p, int64_t count, uint16_t* __restrict__ out) {
  const int per = zeros ? 4 : 2;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < count; i += step) {
    const int j = (int)(i % per), g = (int)(i / per % 8);
    const int64_t grp = i / (per * 8) % groups_p, tile = i / (per * 8) / groups_p;
    const int64_t row = tile * 16 + g + (j & 1) * 8;
    uint16_t v = 0;
    if (row < n && grp < groups) v = (j < 2 ? scales : zeros)[row * groups + grp];
    out[i] = v;
  }
}

// Where a code lies in a 16-bit number, and the bits of 1 around it.
template <typename T>
constexpr int kCodeAt = std::is_same_v<T, __half> ? 6 : 3;
template <typename T>
constexpr uint32_t kOnes = std::is_same_v<T, __half> ? 0x3c003c00u : 0x3f803f80u;

// Pair j of a word: its two codes as (c - 8) / 16.
template <typename T>
__device__ __forceinline__ uint32_t widen2(uint32_t w, int j) {
  using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
  const uint32_t v = ((j ? __funnelshift_r(w, w, 4 * j) : w) & (0x000f000fu << kCodeAt<T>)) | kOnes<T>;
  const uint32_t off = std::is_same_v<T, __half> ? 0x3e003e00u : 0x3fc03fc0u;  // 1.5
  const T2 r = __hsub2(*reinterpret_cast<const T2*>(&v), *reinterpret_cast<const T2*>(&off));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t first_of(uint32_t v) { return v; }
__device__ __forceinline__ uint32_t first_of(uint2 v) { return v.x; }
__device__ __forceinline__ uint32_t second_of(uint32_t) { return 0; }
__device__ __forceinline__ uint32_t second_of(uint2 v) { return v.y; }

// CTAs of a multiprocessor that the registers are held down for
template <int NT>
constexpr int kResident = NT <= 1 ? 4 : NT == 2 ? 3 : NT == 4 ? 2 : 1;

struct Args {
  const uint4* codes;
  const void* scales;
  const void* x;
  const void* bias;
  void* y;
  int64_t sx, sy;
  int32_t n, k, rows, tiles, blocks, groups_p, group_log;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}

// bytes of one stage of a warp's ring: the codes and scales of a block, of MT tiles
template <int MT, bool SUB, bool ZERO>
constexpr int kStage = MT * (512 + (SUB ? 2 : 1) * (ZERO ? 64 : 32));

// A CTA takes MT tiles of 16 outputs by NT*8 rows at a time, and then the next
// ones gridDim.x further on.  Its warps share the blocks of k among them (warp w
// takes blocks w, w + kWarps, ...) and add up at the end, in warp order.  A warp
// copies S blocks ahead, across the tiles' borders too, into a ring of its own
// in shared memory; a lane reads back what it copied itself, but for the scales.
// SUB: groups of 32, two to a block; otherwise a group is whole blocks.
template <typename T, int MT, int NT, int S, bool SUB, bool ZERO>
__global__ void __launch_bounds__(kWarps * 32, kResident<NT>) matvec_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kParts = SUB ? 2 : 1;      // scale groups of a block
  constexpr int kSteps = 4 / kParts;       // matrix steps of a group
  constexpr int kOut = MT * 16;
  constexpr int kSize = kStage<MT, SUB, ZERO>, kScale = ZERO ? 8 : 4;
  using Scale = std::conditional_t<ZERO, uint2, uint32_t>;  // scales (and zero points) of outputs g, g + 8
  float* red = reinterpret_cast<float*>(smem + kWarps * S * kSize);  // [2][warp][row of x][kOut]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int row0 = blockIdx.y * (NT * 8), tile_step = gridDim.x * MT;

  // rows of x past the last one read the last one; their results are dropped
  const T* xp[NT];
#pragma unroll
  for (int j = 0; j < NT; j++)
    xp[j] = reinterpret_cast<const T*>(a.x) + (int64_t)min(row0 + j * 8 + g, a.rows - 1) * a.sx + t * 8;

  // ---- copying ahead
  const unsigned char* ring = smem + warp * (S * kSize);
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  int t_ahead = warp < a.blocks ? blockIdx.x * MT : a.tiles, b_ahead = warp, put = 0;
  auto copy_next = [&]() {
    if (t_ahead < a.tiles) {
#pragma unroll
      for (int m = 0; m < MT; m++) {
        const int tile = min(t_ahead + m, a.tiles - 1);  // a tile past the end repeats the last one
        const uint32_t dst = ring_at + put * kSize;
        copy16(dst + m * 512 + lane * 16, a.codes + ((int64_t)tile * a.blocks + b_ahead) * 32 + lane);
        if (t < kParts) {
          const int grp = SUB ? b_ahead * 2 + t : b_ahead * 64 >> a.group_log;
          copy_small<kScale>(dst + MT * 512 + ((m * kParts + t) * 8 + g) * kScale,
                             reinterpret_cast<const Scale*>(a.scales) + ((int64_t)tile * a.groups_p + grp) * 8 + g);
        }
      }
      b_ahead += kWarps;
      if (b_ahead >= a.blocks) {
        b_ahead = warp;
        t_ahead += tile_step;
      }
      put = put + 1 == S ? 0 : put + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < S - 1; i++) copy_next();

  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int i = 0; i < 4; i++) acc[m][j][i] = 0.f;

  int get = 0, buf = 0;
  for (int tile0 = blockIdx.x * MT; tile0 < a.tiles; tile0 += tile_step) {
    for (int blk = warp; blk < a.blocks; blk += kWarps) {
      uint4 xv[NT][2];
      const bool second = blk * 64 + 32 < a.k;  // k is whole halves of a block
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const uint4* p = reinterpret_cast<const uint4*>(xp[j] + blk * 64);
        xv[j][0] = __ldg(p);
        xv[j][1] = second ? __ldg(p + 4) : make_uint4(0, 0, 0, 0);
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
      __syncwarp();
      copy_next();
      const unsigned char* stage = ring + get * kSize;
      get = get + 1 == S ? 0 : get + 1;
#pragma unroll
      for (int part = 0; part < kParts; part++) {
        float2 sc[MT], off[MT];  // 16 s and (8 - z) s of outputs g and g + 8
#pragma unroll
        for (int m = 0; m < MT; m++) {
          const Scale v = reinterpret_cast<const Scale*>(stage + MT * 512)[(m * kParts + part) * 8 + g];
          sc[m] = unpack2<T>(first_of(v));
          if (ZERO) {
            const float2 z = unpack2<T>(second_of(v));
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
            for (int s = part * kSteps; s < (part + 1) * kSteps; s++) {
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
          const uint4 c = reinterpret_cast<const uint4*>(stage)[m * 32 + lane];
#pragma unroll
          for (int s = part * kSteps; s < (part + 1) * kSteps; s++) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(&c)[s];
            const uint32_t a0 = widen2<T>(w, 0), a1 = widen2<T>(w, 1), a2 = widen2<T>(w, 2), a3 = widen2<T>(w, 3);
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
    // two buffers in turn: a warp can be one tile ahead of the others' reads
    float* part = red + buf * (kWarps * NT * 8 * kOut);
    float* mine = part + warp * (NT * 8 * kOut);
    buf ^= 1;
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          mine[(j * 8 + 2 * t + (i & 1)) * kOut + m * 16 + g + (i >> 1) * 8] = acc[m][j][i];
          acc[m][j][i] = 0.f;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 8 * kOut; i += kWarps * 32) {
      const int r = row0 + i / kOut, n = tile0 * 16 + i % kOut;
      if (r >= a.rows || n >= a.n) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; w++) v += part[w * (NT * 8 * kOut) + i];
      if (a.bias) v += to_f32(reinterpret_cast<const T*>(a.bias)[n]);
      reinterpret_cast<T*>(a.y)[r * a.sy + n] = from_f32<T>(v);
    }
  }
}

template <typename T, int MT, int NT, int S, bool SUB, bool ZERO>
cudaError_t launch(const Args& a, cudaStream_t st) {
  constexpr int smem = kWarps * S * kStage<MT, SUB, ZERO> + 2 * kWarps * NT * 8 * MT * 16 * (int)sizeof(float);
  auto* fn = matvec_kernel<T, MT, NT, S, SUB, ZERO>;
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
  const int rows = (a.rows + NT * 8 - 1) / (NT * 8), tiles = (a.tiles + MT - 1) / MT;
  const int most = (resident * ops_sm_count() + rows - 1) / rows;
  fn<<<dim3(tiles < most ? tiles : most, rows), kWarps * 32, smem, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int MT, int NT, int S>
cudaError_t by_group(const Args& a, bool zeros, cudaStream_t st) {
  if (a.group_log == 5) return zeros ? launch<T, MT, NT, S, true, true>(a, st) : launch<T, MT, NT, S, true, false>(a, st);
  return zeros ? launch<T, MT, NT, S, false, true>(a, st) : launch<T, MT, NT, S, false, false>(a, st);
}

template <typename T>
cudaError_t by_rows(const Args& a, bool zeros, cudaStream_t st) {
  // two tiles of outputs share a CTA's loads of x where that leaves CTAs for
  // every multiprocessor
  const bool two = a.tiles >= 4 * ops_sm_count();
  if (a.rows <= 8) return two ? by_group<T, 2, 1, 4>(a, zeros, st) : by_group<T, 1, 1, 8>(a, zeros, st);
  if (a.rows <= 16) return two ? by_group<T, 2, 2, 4>(a, zeros, st) : by_group<T, 1, 2, 8>(a, zeros, st);
  if (a.rows <= 32) return by_group<T, 2, 4, 4>(a, zeros, st);
  return by_group<T, 2, 8, 4>(a, zeros, st);
}

struct Sizes {
  int64_t tiles, blocks, groups, groups_p, code_bytes, bytes;
};

// NULL, or what is wrong with the matrix's sizes.
const char* sizes(int32_t n, int32_t k, int32_t group, bool zeros, Sizes* s) {
  if (n < 1 || k < 1) return "n and k must be >= 1";
  if (group != 32 && group != 64 && group != 128 && group != 256) return "group must be 32, 64, 128 or 256";
  if (k % group) return "k must be a multiple of group";
  s->tiles = ((int64_t)n + 15) / 16;
  s->blocks = ((int64_t)k + 63) / 64;
  s->groups = k / group;
  s->groups_p = group == 32 ? s->blocks * 2 : s->groups;
  s->code_bytes = s->tiles * s->blocks * 512;
  s->bytes = s->code_bytes + s->tiles * s->groups_p * (zeros ? 64 : 32);
  return nullptr;
}

}  // namespace

int ops_sm_count() {
  static int count[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return 152;
  if (!count[dev]) {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    count[dev] = v > 0 ? v : 152;
  }
  return count[dev];
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
  if (r->rows > 1 && (r->stride_x < 0 || r->stride_y < r->n))
    return api_fail(WFST_ERR_INVALID_ARG, "matvec_quant: stride_y must be >= n and stride_x >= 0");
  if (r->rows > 65535 * 64) return api_fail(WFST_ERR_INVALID_ARG, "matvec_quant: too many rows");
  const int dev = ops_device(r->device, {r->packed, r->x, r->bias, r->y});
  if (dev < 0) return api_fail(WFST_ERR_INVALID_ARG, "matvec_quant: every array must be device memory of one device");
  OpsDevice guard(dev);
  if (guard.err != cudaSuccess) return api_cuda_fail(guard.err, "matvec_quant: device");
  Args a;
  a.codes = reinterpret_cast<const uint4*>(r->packed);
  a.scales = static_cast<const char*>(r->packed) + s.code_bytes;
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
