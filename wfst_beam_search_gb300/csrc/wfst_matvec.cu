// wfst_matvec.cu — products with 4-bit weights.
//
//   y[r, n] = bias[n] + sum_k x[r, k] * s[n, k / G] * (c[n, k] - z[n, k / G])
//
// c are codes 0..15, G the group size, z = 8 where no zero points are given.
// A pass has to read the codes (N*K/2 bytes) and the scales; x and y are small
// beside them, so HBM bounds it up to some tens of rows.
//
// Matrix instructions do the products (m16n8k16: 16 outputs x 8 rows of x),
// also for one row: widening codes to 16 bits and one instruction per 256
// codes leave issue slots free, where products on the general lanes would not.
// The instruction sees the whole numbers c - 8, which the 16-bit types hold
// exactly, with x as it is; a group's fp32 sum is scaled once, so nothing is
// rounded before y.  With zero points the group adds s * (8 - z) * sum x, the
// sum of x coming from the same instruction with ones in place of the codes.
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
#include "wfst_ops.h"

namespace wfst {
namespace {

constexpr int kWarps = 8;
constexpr int kMT = 2;  // 16-output tiles per CTA

// word bits: pair j (0: output g, k 0/1; 1: output g+8, k 0/1; 2: output g,
// k 2/3; 3: output g+8, k 2/3) has its even k at bit 4j, its odd k at 16 + 4j.
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
      uint32_t byte = 0x88;  // code 8 stands for zero past the matrix's edge
      if (row < n && kk < k) byte = codes[row * (k / 2) + kk / 2];
      w |= (byte & 15u) << (4 * j) | (byte >> 4) << (16 + 4 * j);
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

// Codes 0..15 at bits 0-3 and 16-19 of w, as two 16-bit values c - 8 (exact).
template <typename T>
__device__ __forceinline__ uint32_t widen2(uint32_t w);
template <>
__device__ __forceinline__ uint32_t widen2<__half>(uint32_t w) {
  // 1024 + c, less 1032
  const uint32_t v = (w & 0x000f000fu) | 0x64006400u, off = 0x64086408u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&off));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t widen2<__nv_bfloat16>(uint32_t w) {
  // 128 + c, less 136
  const uint32_t v = (w & 0x000f000fu) | 0x43004300u, off = 0x43084308u;
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&off));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t ones2();
template <>
__device__ __forceinline__ uint32_t ones2<__half>() { return 0x3c003c00u; }
template <>
__device__ __forceinline__ uint32_t ones2<__nv_bfloat16>() { return 0x3f803f80u; }

struct Args {
  const uint4* codes;
  const void* scales;
  const void* x;
  const void* bias;
  void* y;
  int64_t sx, sy;
  int32_t n, k, rows, tiles, blocks, groups_p, group;
};

// One CTA: kMT tiles of 16 outputs by NT*8 rows; its warps share the blocks of
// k among them and add up at the end, in warp order.
// SUB: groups of 32, two to a block.  Otherwise a group is whole blocks.
template <typename T, int NT, bool SUB, bool ZERO>
__global__ void __launch_bounds__(kWarps * 32) matvec_kernel(const Args a) {
  extern __shared__ float red[];  // [warp][row of x][kMT * 16 outputs]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int tile0 = blockIdx.x * kMT, row0 = blockIdx.y * (NT * 8);
  constexpr int kParts = SUB ? 2 : 1;      // scale groups of a block
  constexpr int kSteps = 4 / kParts;       // matrix steps of a group
  float acc[kMT][NT][4];
#pragma unroll
  for (int m = 0; m < kMT; m++)
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int i = 0; i < 4; i++) acc[m][j][i] = 0.f;

  for (int blk = warp; blk < a.blocks; blk += kWarps) {
    uint4 c[kMT];
#pragma unroll
    for (int m = 0; m < kMT; m++) {
      const int tile = min(tile0 + m, a.tiles - 1);
      c[m] = __ldcs(a.codes + ((int64_t)tile * a.blocks + blk) * 32 + lane);
    }
    uint4 xv[NT][2];
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const int r = row0 + j * 8 + g;
      const int kk = blk * 64 + t * 8;
      xv[j][0] = xv[j][1] = make_uint4(0, 0, 0, 0);
      if (r < a.rows) {  // k is whole halves of a block
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.x) + r * a.sx + kk);
        xv[j][0] = __ldg(p);
        if (blk * 64 + 32 < a.k) xv[j][1] = __ldg(p + 4);
      }
    }
#pragma unroll
    for (int part = 0; part < kParts; part++) {
      float sum[NT][4];
      if (ZERO) {
#pragma unroll
        for (int j = 0; j < NT; j++) {
          sum[j][0] = sum[j][1] = sum[j][2] = sum[j][3] = 0.f;
#pragma unroll
          for (int s = part * kSteps; s < (part + 1) * kSteps; s++) {
            const uint32_t* xw = reinterpret_cast<const uint32_t*>(xv[j]) + 2 * s;
            mma16816<T>(sum[j], ones2<T>(), ones2<T>(), ones2<T>(), ones2<T>(), xw[0], xw[1]);
          }
        }
      }
      const int grp = SUB ? blk * 2 + part : blk / (a.group / 64);
#pragma unroll
      for (int m = 0; m < kMT; m++) {
        const int tile = min(tile0 + m, a.tiles - 1);
        const int64_t at = ((int64_t)tile * a.groups_p + grp) * 8 + g;
        float2 sc, off = make_float2(0.f, 0.f);
        if (ZERO) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(a.scales) + at);
          sc = unpack2<T>(v.x);
          const float2 z = unpack2<T>(v.y);
          off = make_float2(sc.x * (8.f - z.x), sc.y * (8.f - z.y));
        } else {
          sc = unpack2<T>(__ldg(reinterpret_cast<const uint32_t*>(a.scales) + at));
        }
        float d[NT][4];
#pragma unroll
        for (int j = 0; j < NT; j++) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
#pragma unroll
        for (int s = part * kSteps; s < (part + 1) * kSteps; s++) {
          const uint32_t w = reinterpret_cast<const uint32_t*>(&c[m])[s];
          const uint32_t a0 = widen2<T>(w), a1 = widen2<T>(w >> 4), a2 = widen2<T>(w >> 8), a3 = widen2<T>(w >> 12);
#pragma unroll
          for (int j = 0; j < NT; j++) {
            const uint32_t* xw = reinterpret_cast<const uint32_t*>(xv[j]) + 2 * s;
            mma16816<T>(d[j], a0, a1, a2, a3, xw[0], xw[1]);
          }
        }
#pragma unroll
        for (int j = 0; j < NT; j++) {
          acc[m][j][0] += sc.x * d[j][0];
          acc[m][j][1] += sc.x * d[j][1];
          acc[m][j][2] += sc.y * d[j][2];
          acc[m][j][3] += sc.y * d[j][3];
          if (ZERO) {  // every row of `sum` is the same: its columns 2t, 2t + 1
            acc[m][j][0] += off.x * sum[j][0];
            acc[m][j][1] += off.x * sum[j][1];
            acc[m][j][2] += off.y * sum[j][0];
            acc[m][j][3] += off.y * sum[j][1];
          }
        }
      }
    }
  }

  constexpr int kOut = kMT * 16;
  float* mine = red + (int64_t)warp * (NT * 8 * kOut);
#pragma unroll
  for (int m = 0; m < kMT; m++)
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int i = 0; i < 4; i++) mine[(j * 8 + 2 * t + (i & 1)) * kOut + m * 16 + g + (i >> 1) * 8] = acc[m][j][i];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 8 * kOut; i += kWarps * 32) {
    const int r = row0 + i / kOut, n = tile0 * 16 + i % kOut;
    if (r >= a.rows || n >= a.n) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) v += red[w * (NT * 8 * kOut) + i];
    if (a.bias) v += to_f32(reinterpret_cast<const T*>(a.bias)[n]);
    reinterpret_cast<T*>(a.y)[r * a.sy + n] = from_f32<T>(v);
  }
}

template <typename T, int NT, bool SUB, bool ZERO>
cudaError_t launch(const Args& a, cudaStream_t st) {
  constexpr int smem = kWarps * NT * 8 * kMT * 16 * (int)sizeof(float);
  auto* fn = matvec_kernel<T, NT, SUB, ZERO>;
  static OpsOnce once;
  if (const int dev = ops_current(); smem > 48 * 1024 && !once(dev)) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    once.set(dev);
  }
  const dim3 grid((a.tiles + kMT - 1) / kMT, (a.rows + NT * 8 - 1) / (NT * 8));
  fn<<<grid, kWarps * 32, smem, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int NT>
cudaError_t by_group(const Args& a, bool zeros, cudaStream_t st) {
  if (a.group == 32) return zeros ? launch<T, NT, true, true>(a, st) : launch<T, NT, true, false>(a, st);
  return zeros ? launch<T, NT, false, true>(a, st) : launch<T, NT, false, false>(a, st);
}

template <typename T>
cudaError_t by_rows(const Args& a, bool zeros, cudaStream_t st) {
  if (a.rows <= 8) return by_group<T, 1>(a, zeros, st);
  if (a.rows <= 16) return by_group<T, 2>(a, zeros, st);
  return by_group<T, 4>(a, zeros, st);
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

extern "C" int wfst_quant_pack(const uint8_t* codes, const void* scales, const void* zeros, int32_t n, int32_t k,
                               int32_t group, void* packed, void* stream) {
  Sizes s;
  if (!codes || !scales || !packed) return api_fail(WFST_ERR_INVALID_ARG, "quant_pack: NULL argument");
  if (const char* why = sizes(n, k, group, zeros != nullptr, &s)) return api_fail(WFST_ERR_INVALID_ARG, why);
  if (!aligned(packed, 16)) return api_fail(WFST_ERR_INVALID_ARG, "quant_pack: packed must be 16-byte aligned");
  const int dev = ops_device(-1, {codes, scales, zeros, packed});
  if (dev < 0) return api_fail(WFST_ERR_INVALID_ARG, "quant_pack: every array must be device memory of one device");
  OpsDevice guard(dev);
  if (guard.err != cudaSuccess) return api_cuda_fail(guard.err, "quant_pack: device");
  cudaStream_t st = (cudaStream_t)stream;
  const int grid = ops_sm_count() * 8;
  pack_codes<<<grid, 256, 0, st>>>(codes, n, k, s.blocks, s.code_bytes / 4, reinterpret_cast<uint32_t*>(packed));
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
  if (r->rows > 65535 * 32) return api_fail(WFST_ERR_INVALID_ARG, "matvec_quant: too many rows");
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
  a.group = r->group;
  cudaStream_t st = (cudaStream_t)stream;
  const bool zeros = r->zeros != 0;
  const cudaError_t e =
      r->dtype == WFST_F16 ? by_rows<__half>(a, zeros, st) : by_rows<__nv_bfloat16>(a, zeros, st);
  return e == cudaSuccess ? WFST_OK : api_cuda_fail(e, "matvec_quant launch");
}
