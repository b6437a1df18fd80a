// Root-mean-square norm with the residual's addition in front and the int8
// activation quantisation behind it, and its backward pass.
//
// Forward, one row of k elements:
//   h = RN(x + r),  rstd = RN_fp32(1 / sqrt(mean h^2 + eps)),
//   xn = RN_bf16(RN_fp32(RN_fp32(h rstd) w)),  then the act-quant of xn.
// The row stays in registers between its three uses (the sum of squares, the
// row maximum, the codes), so every operand crosses HBM once.  The squares
// are added in fp64: the result is then the same for every split of the row,
// and rstd is the correctly rounded value but for about one row in 10^7, so
// the int8 codes, which sit behind two roundings, are reproducible.
//
// A row belongs to W warps (one block, or one warp of a block of four rows),
// R vectors of 8 elements a lane.
//
// Measured: forward 4096 x 2560 (fp32 x, bf16 stream, every output) 21.2 us, 5.4
// TB/s; 8192 x 6912 in bf16 to codes 52 us, 5.4 TB/s, where the schedulers issue 58 %
// of the time (18 instructions an element).  Backward 4096 x 2560, three bf16
// gradients, 27.8 us call by call and 27.1 in a graph, 4.5 TB/s (3 us of it the second
// launch); 8191 x 2560 in fp32 68.5 us, 5.5 TB/s; 8192 x 6912 in bf16 75 us.
#include <algorithm>

#include <cuda_bf16.h>

#include "actq_math.cuh"
#include "f32x2.cuh"
#include "sbl_device.cuh"
#include "sbl_kernels.h"

namespace sbl {

namespace {

__device__ __forceinline__ void unpack8(const uint4 a, float (&f)[8]) {
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(u[e] << 16);
    f[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}

template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t vec, float (&f)[8]) {
  if constexpr (F32) {
    const float4* src = static_cast<const float4*>(base) + 2 * vec;
    const float4 a = src[0], b = src[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    unpack8(static_cast<const uint4*>(base)[vec], f);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// RN_fp32(1 / sqrt(a)): the fp32 reciprocal root, two Newton steps in fp64 (the
// second leaves fp64's own rounding errors alone), one rounding.
__device__ __forceinline__ float inverse_root(double a) {
  if (!(a < 1e37)) return static_cast<float>(1.0 / sqrt(a));  // outside fp32, or not finite
  double y = rsqrtf(static_cast<float>(a));
  y = y * (1.5 - 0.5 * a * y * y);
  y = y * (1.5 - 0.5 * a * y * y);
  return static_cast<float>(y);
}

struct NormParams {
  const void *x, *res, *w;
  int64_t t;
  int nvec;  // k / 8
  double inv_k, eps;
  int w_f32;
  void* h;
  uint4 *xn, *xhat;
  uint2* xq;
  float *xscale, *rstd;
  uint32_t* status;
};

// Residual types of the forward kernel.
enum { kNoRes = 0, kResBf16 = 1, kResF32 = 2 };

__device__ __forceinline__ f32x2 unpack2(uint32_t w) {
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(f32x2 v) {
  const float2 f = halves(v);
  return pack2(f.x, f.y);
}

// The larger magnitudes of two pairs of bf16 values; a NaN stays.
__device__ __forceinline__ uint32_t top2(uint32_t top, uint32_t w) {
  const __nv_bfloat162 a = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&top),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&a);
}

// Eight elements as they lie in memory.
template <bool F32>
struct Raw {
  uint4 w[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t vec) {
    const uint4* src = static_cast<const uint4*>(base) + (F32 ? 2 : 1) * vec;
    w[0] = src[0];
    if constexpr (F32) w[1] = src[1];
  }
  __device__ __forceinline__ void zero() {
    w[0] = make_uint4(0, 0, 0, 0);
    if constexpr (F32) w[1] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void unpack(f32x2 (&f)[4]) const {
    if constexpr (F32) {
      f[0] = pair(__uint_as_float(w[0].x), __uint_as_float(w[0].y));
      f[1] = pair(__uint_as_float(w[0].z), __uint_as_float(w[0].w));
      f[2] = pair(__uint_as_float(w[1].x), __uint_as_float(w[1].y));
      f[3] = pair(__uint_as_float(w[1].z), __uint_as_float(w[1].w));
    } else {
      f[0] = unpack2(w[0].x), f[1] = unpack2(w[0].y), f[2] = unpack2(w[0].z), f[3] = unpack2(w[0].w);
    }
  }
};

__device__ __forceinline__ uint4 pack8(const f32x2 (&f)[4]) {
  return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}

// Eight codes as quantise8_fma gives them, and the bf16 values they stand for:
// the code is at hand as a float (its byte's sum minus 1.5 2^23), so no byte is
// taken apart again.
__device__ __forceinline__ uint2 quantise8_values(const uint4 v, float c, float a_over_127, uint4* values) {
  const uint32_t words[4] = {v.x, v.y, v.z, v.w};
  const f32x2 c2 = pair(c, c), a2 = pair(a_over_127, a_over_127), up = pair(12582912.0f, 12582912.0f),
              down = pair(-12582912.0f, -12582912.0f);
  uint32_t bytes[4], packed[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const f32x2 f = fma2(unpack2(words[h]), c2, up);
    const float2 b = halves(f);
    bytes[h] = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
    packed[h] = pack2(mul2(add2(f, down), a2));
  }
  *values = make_uint4(packed[0], packed[1], packed[2], packed[3]);
  return make_uint2(__byte_perm(bytes[0], bytes[1], 0x5410), __byte_perm(bytes[2], bytes[3], 0x5410));
}

constexpr int kNormMaxWarps = 16;  // of a row with few rows at hand
constexpr int kNormRowWarps = 12;  // of a row otherwise (with a residual: 168 registers a thread at most)

// A block walks rows with a stride of the grid; the next row's loads are on
// their way while a row is computed.  The weight lies in shared memory as fp32
// for all of the block's rows, or (FEW: a block has one row) is loaded beside it.
template <bool XF32, int RES, int R, bool ONE_WARP, bool FEW>
__global__ void __launch_bounds__(ONE_WARP ? 128 : 32 * (FEW || RES == kNoRes ? kNormMaxWarps : kNormRowWarps), 1)
    k_rmsnorm(const NormParams p) {
  constexpr bool HF32 = RES == kNoRes ? XF32 : RES == kResF32;
  __shared__ double s_sum[2][kNormMaxWarps];
  __shared__ uint32_t s_max[2][kNormMaxWarps];
  extern __shared__ float4 s_w[];  // [k / 4], without FEW
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = ONE_WARP ? 1 : static_cast<int>(blockDim.x) / 32;
  const bool first = ONE_WARP ? lane == 0 : threadIdx.x == 0;
  // a warp's vectors lie side by side: their offsets are constants
  const int at = (ONE_WARP ? 0 : warp * R * 32) + lane;
  constexpr int kRows = ONE_WARP ? 4 : 1;
  int64_t row = ONE_WARP ? int64_t(blockIdx.x) * kRows + warp : int64_t(blockIdx.x);
  pdl_wait();
  pdl_trigger();

  Raw<XF32> x[R];
  Raw<RES == kResF32> q[RES == kNoRes ? 1 : R];
  const auto fetch = [&](int64_t next) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = at + r * 32;
      if (i < p.nvec) {
        x[r].load(p.x, next * p.nvec + at + r * 32);
        if constexpr (RES != kNoRes) q[r].load(p.res, next * p.nvec + at + r * 32);
      }
    }
  };
#pragma unroll
  for (int r = 0; r < R; ++r) {  // lanes past the row's end hold zeros throughout
    x[r].zero();
    if constexpr (RES != kNoRes) q[r].zero();
  }
  if (row < p.t) fetch(row);
  f32x2 w[FEW ? R : 1][4];
  if (p.w != nullptr) {
    if constexpr (FEW) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = at + r * 32;
        if (i >= p.nvec) continue;
        if (p.w_f32) {
          Raw<true> u;
          u.load(p.w, i);
          u.unpack(w[r]);
        } else {
          Raw<false> u;
          u.load(p.w, i);
          u.unpack(w[r]);
        }
      }
    } else {
      for (int i = threadIdx.x; i < p.nvec; i += blockDim.x) {
        float f[8];
        if (p.w_f32)
          load8<true>(p.w, i, f);
        else
          load8<false>(p.w, i, f);
        s_w[2 * i] = make_float4(f[0], f[1], f[2], f[3]);
        s_w[2 * i + 1] = make_float4(f[4], f[5], f[6], f[7]);
      }
      __syncthreads();
    }
  }
  const bool quant = p.xhat != nullptr || p.xq != nullptr || p.xscale != nullptr;

  for (int parity = 0; row < p.t; parity ^= 1) {
    const int64_t base = row * p.nvec + at, next = row + int64_t(gridDim.x) * kRows;
    f32x2 h[R][4];
    double ss[2] = {0.0, 0.0};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = at + r * 32;
      x[r].unpack(h[r]);
      if constexpr (RES != kNoRes) {
        f32x2 u[4];
        q[r].unpack(u);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[r][e] = add2(h[r][e], u[e]);
      }
      if constexpr (HF32) {
        if (p.h != nullptr && i < p.nvec) {
          const float2 a = halves(h[r][0]), b = halves(h[r][1]), c = halves(h[r][2]), d = halves(h[r][3]);
          float4* dst = static_cast<float4*>(p.h) + 2 * (base + r * 32);
          dst[0] = make_float4(a.x, a.y, b.x, b.y);
          dst[1] = make_float4(c.x, c.y, d.x, d.y);
        }
      } else if constexpr (RES != kNoRes || XF32) {
        const uint4 b = pack8(h[r]);
        if (p.h != nullptr && i < p.nvec) static_cast<uint4*>(p.h)[base + r * 32] = b;
        h[r][0] = unpack2(b.x), h[r][1] = unpack2(b.y), h[r][2] = unpack2(b.z), h[r][3] = unpack2(b.w);
      } else {
        if (p.h != nullptr && i < p.nvec) static_cast<uint4*>(p.h)[base + r * 32] = x[r].w[0];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = halves(h[r][e]);
        const double a = f.x, b = f.y;
        ss[0] = fma(a, a, ss[0]);
        ss[1] = fma(b, b, ss[1]);
      }
    }
    if (!FEW && next < p.t) fetch(next);
    double sum = ss[0] + ss[1];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (!ONE_WARP) {
      if (lane == 0) s_sum[parity][warp] = sum;
      __syncthreads();
      sum = s_sum[parity][0];
      for (int i = 1; i < warps; ++i) sum += s_sum[parity][i];
    }
    const float rstd = inverse_root(fma(sum, p.inv_k, p.eps));
    if (first) {
      if (p.rstd != nullptr) p.rstd[row] = rstd;
      if (!(sum < __longlong_as_double(0x7FF0000000000000ll))) raise_status(p.status, SBL_STATUS_NONFINITE_X);
    }
    if (p.xn != nullptr || quant) {
      uint4 v[R];
      uint32_t m2 = 0;
      const f32x2 rstd2 = pair(rstd, rstd);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = at + r * 32;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[r][e] = mul2(h[r][e], rstd2);
        if (p.w != nullptr && i < p.nvec) {
          if constexpr (FEW) {
#pragma unroll
            for (int e = 0; e < 4; ++e) h[r][e] = mul2(h[r][e], w[r][e]);
          } else {
            const float4 a = s_w[2 * i], b = s_w[2 * i + 1];
            h[r][0] = mul2(h[r][0], pair(a.x, a.y)), h[r][1] = mul2(h[r][1], pair(a.z, a.w));
            h[r][2] = mul2(h[r][2], pair(b.x, b.y)), h[r][3] = mul2(h[r][3], pair(b.z, b.w));
          }
        }
        v[r] = pack8(h[r]);
        if (p.xn != nullptr && i < p.nvec) p.xn[base + r * 32] = v[r];
        m2 = top2(m2, v[r].x);
        m2 = top2(m2, v[r].y);
        m2 = top2(m2, v[r].z);
        m2 = top2(m2, v[r].w);
      }
      uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
      if (m >= 0x7F80u) raise_status(p.status, SBL_STATUS_NONFINITE_X);
      if (quant) {
        m = __reduce_max_sync(0xffffffffu, m);
        if constexpr (!ONE_WARP) {
          if (lane == 0) s_max[parity][warp] = m;
          __syncthreads();
          m = s_max[parity][0];
          for (int i = 1; i < warps; ++i) m = max(m, s_max[parity][i]);
        }
        const float ap = fmaxf(__uint_as_float(m << 16), 1e-5f);
        if (first && p.xscale != nullptr) p.xscale[row] = ap;
        const QScale qs = make_qscale(ap);
        const bool zeros = m == 0;  // padding: no division for it
        const float a_over_127 = __fdiv_rn(ap, 127.0f);
        if (qs.exact && !zeros) {  // the clamp or a' >= 2^120: the IEEE division
#pragma unroll 1
          for (int r = 0; r < R; ++r) {
            const int i = at + r * 32;
            if (i >= p.nvec) break;
            uint4 u = v[0];  // v[r], without a register array indexed at run time
#pragma unroll
            for (int j = 1; j < R; ++j)
              if (j == r) u = v[j];
            if (p.xq != nullptr) p.xq[base + r * 32] = quantise8_div(u, ap);
            if (p.xhat != nullptr) p.xhat[base + r * 32] = dequantise8(u, qs);
          }
        } else {  // one multiply-add a code; zeros give zeros
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const int i = at + r * 32;
            if (i < p.nvec) {
              uint4 values;
              const uint2 c = quantise8_values(v[r], qs.c, a_over_127, &values);
              if (p.xq != nullptr) p.xq[base + r * 32] = c;
              if (p.xhat != nullptr) p.xhat[base + r * 32] = values;
            }
          }
        }
      }
    }
    if (FEW) break;
    row = next;
  }
}

template <bool XF32, int RES, int R, bool ONE_WARP, bool FEW>
cudaError_t launch_norm(const NormParams& p, int warps, int num_sms, cudaStream_t s) {
  constexpr int rows = ONE_WARP ? 4 : 1;
  const int threads = ONE_WARP ? 128 : 32 * warps;
  const size_t smem = !FEW && p.w != nullptr ? size_t(p.nvec) * 32 : 0;
  int64_t blocks = (p.t + rows - 1) / rows;
  if constexpr (!FEW) {
    // one wave of blocks, each with its share of the rows
    int fit = 0;
    cudaError_t e = cudaSuccess;
    if (smem > 40 * 1024)  // with the static arrays past the 48 KB that need no asking; the same for every size:
                           // another thread's call may come between this one's asking and its launch
      e = cudaFuncSetAttribute(k_rmsnorm<XF32, RES, R, ONE_WARP, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               SBL_NORM_MAX_K * 4);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, k_rmsnorm<XF32, RES, R, ONE_WARP, FEW>, threads, smem);
    if (e != cudaSuccess) return e;
    blocks = std::min<int64_t>(blocks, int64_t(std::max(fit, 1)) * num_sms);
  }
  return launch_pdl(k_rmsnorm<XF32, RES, R, ONE_WARP, FEW>, dim3(static_cast<unsigned>(blocks)), dim3(threads), smem, s,
                    p);
}

template <bool XF32, int RES, int R>
cudaError_t launch_norm(const NormParams& p, int warps, bool few, int num_sms, cudaStream_t s) {
  if constexpr (R <= 4)
    if (few) return launch_norm<XF32, RES, R, false, true>(p, warps, num_sms, s);
  if (warps == 1) return launch_norm<XF32, RES, R, true, false>(p, warps, num_sms, s);
  return launch_norm<XF32, RES, R, false, false>(p, warps, num_sms, s);
}

// Warps a row and vectors a lane.  Every warp repeats the row's scalar work (the
// root, the quantiser's constants: some 200 instructions).  Without a residual
// that issue is the bound and a lane takes many vectors (8192 x 6912 in bf16:
// 7 a lane 50 us, 6: 56, 3: 65); with one, more bytes arrive for the same
// arithmetic and more rows in flight count (4096 x 2560, fp32 on a bf16 stream:
// 2 a lane 19.3 us, 3: 20.2, 5: 19.9; 8192 x 4096 in bf16: 2 a lane 50 us, 4: 57).
// Up to three vectors less where that leaves fewer lanes idle.  With few rows the row's
// own latency counts and more warps share it (one row of 2560: 2.3 against 3.4 us).
template <bool XF32, int RES>
cudaError_t pick_norm(const NormParams& p, int num_sms, cudaStream_t s) {
  const int n = p.nvec;
  const bool few = p.t <= 2 * num_sms;
  const auto up = [](int a, int b) { return (a + b - 1) / b; };
  int warps = std::min(up(n, 32), kNormMaxWarps);
  if (!few) {
    const int most = std::max(RES != kNoRes ? 2 : XF32 ? 5 : 7, up(n, 32 * kNormRowWarps));
    warps = up(n, 32 * most);
    for (int r = most - 1; r >= std::max(most - 3, 1); --r) {
      const int w = up(n, 32 * r);
      if (w <= kNormRowWarps && w * up(n, 32 * w) < warps * up(n, 32 * warps)) warps = w;
    }
  }
  switch (up(n, 32 * warps)) {
    case 1: return launch_norm<XF32, RES, 1>(p, warps, few, num_sms, s);
    case 2: return launch_norm<XF32, RES, 2>(p, warps, few, num_sms, s);
    case 3: return launch_norm<XF32, RES, 3>(p, warps, few, num_sms, s);
    case 4: return launch_norm<XF32, RES, 4>(p, warps, few, num_sms, s);
    case 5: return launch_norm<XF32, RES, 5>(p, warps, few, num_sms, s);
    case 6: return launch_norm<XF32, RES, 6>(p, warps, few, num_sms, s);
    default: break;
  }
  if constexpr (!XF32 && RES == kNoRes) return launch_norm<XF32, RES, 7>(p, warps, few, num_sms, s);
  return cudaErrorInvalidValue;  // not reached: k is at most SBL_NORM_MAX_K
}

// ---------------------------------------------------------------------------
// Backward: g = sum dy, n = h rstd, c = mean(w g n),
//   dh = dres + rstd (w g - n c),   dw = sum over rows of g n.
// A group of warps walks rows with a fixed stride and keeps its columns' share
// of dw in registers.  Up to five arrays are read for one written: each thread
// copies its own vectors of the rows to come into its own slots of shared memory
// (cp.async, a ring of `depth` rows a group), which costs no registers and needs no
// barrier, since no other thread reads them.  The groups of a block add their dw in
// shared memory in a fixed order, one row of partial sums a block goes to the
// workspace, and a second launch adds those, in a fixed order too.
// What bounds 4096 x 2560 with three gradients is a row's chain: some 890
// instructions a warp and row on 8 warps an SM, seven rows in turn, the schedulers
// issuing 33 % of the time, with 200 KB an SM on their way; one row more in the ring
// gains nothing.  fp32 rows are bound by HBM.
// ---------------------------------------------------------------------------
struct NormBwdParams {
  const void* h;
  const float* rstd;
  const void* w;
  const void* dy[3];
  int ndy;
  const void* dres;
  int64_t t;
  int nvec;
  float inv_k;
  int w_f32;
  int warps, groups;  // warps a row, rows a block at a time
  int depth, words;   // rows of the ring (1 to 3), 16-byte words a thread and row
  void* dh;
  void* dx;
  float* part;  // [gridDim.x][k], or nullptr without dw
};

constexpr int kNormBwdThreads = 512, kNormBwdRuns = 5;  // of a block; runs of 256 elements a warp at most
constexpr int kNormBwdSmem = 224 * 1024;                // dynamic shared memory of a block at most

template <int BYTES>
__device__ __forceinline__ void copy_async(void* smem, const void* gmem) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(gmem) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(smem)), "l"(gmem), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The eight elements of a lane in a run of 256.  Where an array is fp32 (QUADS)
// they are two quads 128 elements apart, so that the warp's 16-byte accesses lie
// side by side (asynchronous copies do not pass through L1: two accesses to the
// halves of a sector would fetch it twice, 99 us instead of 68 at 8191 x 2560);
// with bf16 alone they are eight in a row.  `in`: which of the lane's quads lie
// in the row (without QUADS both or none).
template <bool F32, bool QUADS>
__device__ __forceinline__ void copy8_async(uint4* dst, const void* base, int64_t el, bool in0, bool in1) {
  const float* f = static_cast<const float*>(base) + el;
  const uint16_t* h = static_cast<const uint16_t*>(base) + el;
  if constexpr (F32) {
    if (in0) copy_async<16>(dst, f);
    if (in1) copy_async<16>(dst + 32, f + 128);
  } else if constexpr (QUADS) {
    if (in0) copy_async<8>(dst, h);
    if (in1) copy_async<8>(reinterpret_cast<uint2*>(dst) + 1, h + 128);
  } else {
    if (in0) copy_async<16>(dst, h);
  }
}

template <bool F32, bool QUADS>
__device__ __forceinline__ Raw<F32> load8_at(const void* base, int64_t el, bool in0, bool in1) {
  const float* f = static_cast<const float*>(base) + el;
  const uint16_t* h = static_cast<const uint16_t*>(base) + el;
  Raw<F32> u;
  u.zero();
  if constexpr (F32) {
    if (in0) u.w[0] = *reinterpret_cast<const uint4*>(f);
    if (in1) u.w[1] = *reinterpret_cast<const uint4*>(f + (QUADS ? 128 : 4));
  } else if constexpr (QUADS) {
    uint2 a = make_uint2(0, 0), b = make_uint2(0, 0);
    if (in0) a = *reinterpret_cast<const uint2*>(h);
    if (in1) b = *reinterpret_cast<const uint2*>(h + 128);
    u.w[0] = make_uint4(a.x, a.y, b.x, b.y);
  } else {
    if (in0) u.w[0] = *reinterpret_cast<const uint4*>(h);
  }
  return u;
}

template <bool QUADS>
__device__ __forceinline__ void store8_bf16(void* base, int64_t el, const uint4 b, bool in0, bool in1) {
  uint16_t* dst = static_cast<uint16_t*>(base) + el;
  if constexpr (QUADS) {
    if (in0) *reinterpret_cast<uint2*>(dst) = make_uint2(b.x, b.y);
    if (in1) *reinterpret_cast<uint2*>(dst + 128) = make_uint2(b.z, b.w);
  } else {
    if (in0) *reinterpret_cast<uint4*>(dst) = b;
  }
}

template <bool HF32, bool DF32, int R, bool RING>
__global__ void __launch_bounds__(kNormBwdThreads, 1) k_rmsnorm_bwd(const NormBwdParams p) {
  constexpr int HW = HF32 ? 2 : 1, DW = DF32 ? 2 : 1;
  constexpr bool QUADS = HF32 || DF32;
  extern __shared__ uint4 s_ring[];
  __shared__ float s_part[2][kNormBwdThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / p.warps, k = 8 * p.nvec;
  const int at = (warp - group * p.warps) * R * 256 + (QUADS ? 4 : 8) * lane;
  const int64_t first = blockIdx.x + int64_t(group) * gridDim.x, stride = int64_t(p.groups) * gridDim.x;
  bool in0[R], in1[R];
#pragma unroll
  for (int r = 0; r < R; ++r) in0[r] = at + r * 256 < k, in1[r] = at + r * 256 + (QUADS ? 128 : 0) < k;
  pdl_wait();
  pdl_trigger();

  // A warp's slot holds the words of its part of a row, 32 lanes each: h, dres,
  // the gradients, R runs of each; so every word has a constant offset.
  constexpr int kRes = R * HW, kDy = 2 * R * HW, kOne = R * DW;
  uint4* const mine = s_ring + warp * p.depth * p.words * 32 + lane;
  const int slot_step = p.words * 32;
  const auto fetch = [&](int64_t row, uint4* dst) {
    const int64_t el = row * k + at;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      copy8_async<HF32, QUADS>(dst + r * HW * 32, p.h, el + r * 256, in0[r], in1[r]);
      if (p.dres != nullptr)
        copy8_async<HF32, QUADS>(dst + (kRes + r * HW) * 32, p.dres, el + r * 256, in0[r], in1[r]);
#pragma unroll
      for (int d = 0; d < 3; ++d)
        if (d < p.ndy)
          copy8_async<DF32, QUADS>(dst + (kDy + d * kOne + r * DW) * 32, p.dy[d], el + r * 256, in0[r], in1[r]);
    }
  };
  // Run r of an array: out of the slot (its word), or (RING false) out of memory.
  const auto h_at = [&](const uint4* src, int word, const void* base, int64_t el, int r) {
    if constexpr (RING) {
      Raw<HF32> u;
#pragma unroll
      for (int j = 0; j < HW; ++j) u.w[j] = src[(word + r * HW + j) * 32];
      return u;
    } else {
      return load8_at<HF32, QUADS>(base, el + r * 256, in0[r], in1[r]);
    }
  };
  const auto d_at = [&](const uint4* src, int word, const void* base, int64_t el, int r) {
    if constexpr (RING) {
      Raw<DF32> u;
#pragma unroll
      for (int j = 0; j < DW; ++j) u.w[j] = src[(word + r * DW + j) * 32];
      return u;
    } else {
      return load8_at<DF32, QUADS>(base, el + r * 256, in0[r], in1[r]);
    }
  };
  if constexpr (RING)  // words that no copy fills (past the row's end) stay zero
    for (int i = 0; i < p.depth * p.words; ++i) mine[i * 32] = make_uint4(0, 0, 0, 0);
  float* const s_w = reinterpret_cast<float*>(s_ring + (blockDim.x >> 5) * p.depth * p.words * 32);
  if constexpr (RING)
    if (p.w != nullptr) {
      for (int i = threadIdx.x; i < p.warps * R * 32; i += blockDim.x) {
        float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (i < p.nvec) {
          if (p.w_f32)
            load8<true>(p.w, i, f);
          else
            load8<false>(p.w, i, f);
        }
        *reinterpret_cast<float4*>(s_w + 8 * i) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(s_w + 8 * i + 4) = make_float4(f[4], f[5], f[6], f[7]);
      }
    }

  f32x2 acc[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[r][e] = pair(0.0f, 0.0f);
  if constexpr (RING) {
    int64_t row = first;
    for (int d = 0; d < p.depth; ++d, row += stride) {
      if (row < p.t) fetch(row, mine + d * slot_step);
      copy_commit();
    }
  }
  if constexpr (RING) __syncthreads();  // the weight

  int slot = 0, parity = 0;
  float rstd_next = first < p.t ? p.rstd[first] : 0.0f;
  for (int64_t row = first; row < p.t; row += stride) {
    const int64_t el = row * k + at;
    const float rstd = rstd_next;
    if (row + stride < p.t) rstd_next = p.rstd[row + stride];
    if constexpr (RING) {
      if (p.depth == 3)
        copy_wait<2>();
      else if (p.depth == 2)
        copy_wait<1>();
      else
        copy_wait<0>();
    }
    uint4* const src = mine + slot * slot_step;
    const f32x2 rstd2 = pair(rstd, rstd);
    f32x2 g[R][4], c2 = pair(0.0f, 0.0f);  // n is formed again below: its registers hold more rows instead
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f32x2 u[4], n[4];
      h_at(src, 0, p.h, el, r).unpack(n);
      d_at(src, kDy, p.dy[0], el, r).unpack(g[r]);
      if (p.ndy > 1) {
        d_at(src, kDy + kOne, p.dy[1], el, r).unpack(u);
#pragma unroll
        for (int e = 0; e < 4; ++e) g[r][e] = add2(g[r][e], u[e]);
      }
      if (p.ndy > 2) {
        d_at(src, kDy + 2 * kOne, p.dy[2], el, r).unpack(u);
#pragma unroll
        for (int e = 0; e < 4; ++e) g[r][e] = add2(g[r][e], u[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        n[e] = mul2(n[e], rstd2);
        acc[r][e] = fma2(g[r][e], n[e], acc[r][e]);
      }
      if (p.w != nullptr) {
        if constexpr (RING) {
          const float4* w = reinterpret_cast<const float4*>(s_w + at + r * 256);
          const float4 a = w[0], b = w[QUADS ? 32 : 1];
          u[0] = pair(a.x, a.y), u[1] = pair(a.z, a.w), u[2] = pair(b.x, b.y), u[3] = pair(b.z, b.w);
        } else if (p.w_f32) {
          load8_at<true, QUADS>(p.w, at + r * 256, in0[r], in1[r]).unpack(u);
        } else {
          load8_at<false, QUADS>(p.w, at + r * 256, in0[r], in1[r]).unpack(u);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) g[r][e] = mul2(g[r][e], u[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) c2 = fma2(g[r][e], n[e], c2);
    }
    const float2 ch = halves(c2);
    float c = ch.x + ch.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (p.warps > 1) {
      if (lane == 0) s_part[parity][warp] = c;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(p.warps * 32) : "memory");
      c = (lane & 15) < p.warps ? s_part[parity][group * p.warps + (lane & 15)] : 0.0f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
      parity ^= 1;  // a place is written again two rows on, behind another barrier
    }
    c *= -p.inv_k;
    const f32x2 minus = pair(c, c);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f32x2 d[4], n[4];
      h_at(src, 0, p.h, el, r).unpack(n);
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = mul2(rstd2, fma2(mul2(n[e], rstd2), minus, g[r][e]));
      if (p.dres != nullptr) {
        f32x2 u[4];
        h_at(src, kRes, p.dres, el, r).unpack(u);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = add2(d[e], u[e]);
      }
      const uint4 b = pack8(d);
      if constexpr (HF32) {
        const float2 d0 = halves(d[0]), d1 = halves(d[1]), d2 = halves(d[2]), d3 = halves(d[3]);
        float* dst = static_cast<float*>(p.dh) + el + r * 256;
        if (in0[r]) *reinterpret_cast<float4*>(dst) = make_float4(d0.x, d0.y, d1.x, d1.y);
        if (in1[r]) *reinterpret_cast<float4*>(dst + 128) = make_float4(d2.x, d2.y, d3.x, d3.y);
      } else {
        store8_bf16<QUADS>(p.dh, el + r * 256, b, in0[r], in1[r]);
      }
      if (p.dx != nullptr) store8_bf16<QUADS>(p.dx, el + r * 256, b, in0[r], in1[r]);
    }
    if constexpr (RING) {  // this row's slot is read: the copies of a row to come may take it
      const int64_t later = row + p.depth * stride;
      if (later < p.t) fetch(later, src);
      copy_commit();
      if (++slot == p.depth) slot = 0;
    }
  }
  if (p.part == nullptr) return;
  // the groups' shares side by side, then added in the groups' order
  float* const dst = p.part + int64_t(blockIdx.x) * k;
  float* const share = p.groups > 1 ? reinterpret_cast<float*>(s_ring) + group * k : dst;
  copy_wait<0>();
  if (p.groups > 1) __syncthreads();  // every group is done with the ring
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (!(q ? in1[r] : in0[r])) continue;
      const float2 a0 = halves(acc[r][2 * q]), a1 = halves(acc[r][2 * q + 1]);
      *reinterpret_cast<float4*>(share + at + r * 256 + q * (QUADS ? 128 : 4)) = make_float4(a0.x, a0.y, a1.x, a1.y);
    }
  if (p.groups == 1) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.nvec; i += blockDim.x) {
    const float4* src = reinterpret_cast<const float4*>(s_ring) + i;
    float4 a = src[0];
    for (int g = 1; g < p.groups; ++g) {
      const float4 b = src[g * 2 * p.nvec];
      a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
    }
    reinterpret_cast<float4*>(dst)[i] = a;
  }
}

// dw[c] = sum of the blocks' partial sums: 8 threads of 4 columns across, 32
// rows of partial sums beside each other (at most 8 each, all loads at once),
// then a tree over the 32.
__global__ void __launch_bounds__(256) k_norm_dw(const float4* __restrict__ part, int blocks, int n4, float4* dw) {
  __shared__ float4 s[32][8];
  pdl_wait();
  pdl_trigger();
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int col = blockIdx.x * 8 + x;
  float4 a = make_float4(0, 0, 0, 0);
  if (col < n4) {
    float4 v[kNormBwdMaxBlocks / 32];
#pragma unroll
    for (int i = 0; i < kNormBwdMaxBlocks / 32; ++i) {
      const int b = y + 32 * i;
      v[i] = b < blocks ? __ldcg(part + int64_t(b) * n4 + col) : make_float4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kNormBwdMaxBlocks / 32; ++i) a.x += v[i].x, a.y += v[i].y, a.z += v[i].z, a.w += v[i].w;
  }
  s[y][x] = a;
  __syncthreads();
  if (y >= 4) return;  // one warp: four rows of eight columns
  for (int i = y + 4; i < 32; i += 4) {
    const float4 v = s[i][x];
    a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    a.x += __shfl_down_sync(0xffffffffu, a.x, o), a.y += __shfl_down_sync(0xffffffffu, a.y, o);
    a.z += __shfl_down_sync(0xffffffffu, a.z, o), a.w += __shfl_down_sync(0xffffffffu, a.w, o);
  }
  if (y == 0 && col < n4) dw[col] = a;
}

template <bool HF32, bool DF32, int R, bool RING>
cudaError_t launch_norm_bwd(const NormBwdParams& p, int blocks, size_t smem, cudaStream_t s) {
  // the same for every size: another thread's call may come between this and the launch
  const cudaError_t e = cudaFuncSetAttribute(k_rmsnorm_bwd<HF32, DF32, R, RING>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kNormBwdSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_rmsnorm_bwd<HF32, DF32, R, RING>, dim3(blocks), dim3(32 * p.warps * p.groups), smem, s, p);
}

// Warps a row and runs a warp: the fewest instructions for a row, of which a
// warp spends some 180 beside 160 a run (8192 x 6912 in bf16: 7 warps of 4 runs
// 75.5 us, 14 of 2 runs 126).  As many rows at a time as 14 warps hold, with the
// most of them in the ring, but no more than there are rows for all SMs; one
// block an SM.  The two warps' registers that are left hold blocks of the second
// launch, which then start at once (4096 x 2560, three gradients, in a graph: 28.2 ->
// 27.1 us).
template <bool HF32, bool DF32>
cudaError_t pick_norm_bwd(NormBwdParams p, float* dw, int num_sms, cudaStream_t s) {
  constexpr int most_warps = kNormBwdThreads / 32;
  const auto up = [](int a, int b) { return (a + b - 1) / b; };
  p.warps = up(p.nvec, 32 * kNormBwdRuns);
  for (int w = p.warps + 1; w <= most_warps; ++w)
    if (w * (180 + 160 * up(p.nvec, 32 * w)) < p.warps * (180 + 160 * up(p.nvec, 32 * p.warps))) p.warps = w;
  const int r = up(p.nvec, 32 * p.warps);
  p.words = r * ((HF32 ? 2 : 1) * 2 + (DF32 ? 2 : 1) * p.ndy);
  const size_t weight = p.w != nullptr ? size_t(p.warps) * r * 1024 : 0;  // fp32, behind the ring
  const size_t room = kNormBwdSmem - weight;
  const size_t one = size_t(p.words) * 16 * 32 * p.warps;
  const auto depth = [&](int groups) { return static_cast<int>(std::min<size_t>(room / (one * groups), 3)); };
  const int most = static_cast<int>(std::min<int64_t>({std::max(14 / p.warps, 1), (p.t + num_sms - 1) / num_sms}));
  p.groups = most;
  for (int g = most - 1; g >= 1; --g)
    if (g * depth(g) > p.groups * depth(p.groups)) p.groups = g;
  p.depth = depth(p.groups);
  const size_t smem = std::max<size_t>(p.depth > 0 ? p.depth * one * p.groups + weight : 0,
                                       p.groups > 1 ? size_t(p.groups) * p.nvec * 32 : 0);  // 80 KB at most
  const int blocks = static_cast<int>(std::min<int64_t>(p.t, num_sms));
  cudaError_t e;
  if (p.depth == 0)  // not even one row fits: long fp32 rows of several arrays
    e = launch_norm_bwd<HF32, DF32, kNormBwdRuns, false>(p, blocks, smem, s);
  else if (r == 1)
    e = launch_norm_bwd<HF32, DF32, 1, true>(p, blocks, smem, s);
  else if (r == 2)
    e = launch_norm_bwd<HF32, DF32, 2, true>(p, blocks, smem, s);
  else if (r == 3)
    e = launch_norm_bwd<HF32, DF32, 3, true>(p, blocks, smem, s);
  else if (r == 4)
    e = launch_norm_bwd<HF32, DF32, 4, true>(p, blocks, smem, s);
  else
    e = launch_norm_bwd<HF32, DF32, 5, true>(p, blocks, smem, s);
  if (e != cudaSuccess || dw == nullptr) return e;
  const int n4 = 2 * p.nvec;
  return launch_pdl(k_norm_dw, dim3((n4 + 7) / 8), dim3(256), 0, s, reinterpret_cast<const float4*>(p.part), blocks,
                    n4, reinterpret_cast<float4*>(dw));
}

}  // namespace

cudaError_t launch_rmsnorm(const sbl_rmsnorm_args& a, int num_sms, cudaStream_t s) {
  NormParams p;
  p.x = a.x, p.res = a.residual, p.w = a.weight;
  p.t = a.t, p.nvec = static_cast<int>(a.k / 8);
  p.inv_k = 1.0 / static_cast<double>(a.k), p.eps = a.eps;
  p.w_f32 = (a.flags & SBL_NORM_W_F32) != 0u;
  p.h = a.h_out;
  p.xn = static_cast<uint4*>(a.xn_out), p.xhat = static_cast<uint4*>(a.xhat_out);
  p.xq = reinterpret_cast<uint2*>(a.xq_out);
  p.xscale = a.xscale_out, p.rstd = a.rstd_out, p.status = a.status_dev;
  const bool xf = (a.flags & SBL_NORM_X_F32) != 0u, rf = (a.flags & SBL_NORM_STREAM_F32) != 0u;
  if (a.residual == nullptr)
    return xf ? pick_norm<true, kNoRes>(p, num_sms, s) : pick_norm<false, kNoRes>(p, num_sms, s);
  if (rf) return xf ? pick_norm<true, kResF32>(p, num_sms, s) : pick_norm<false, kResF32>(p, num_sms, s);
  return xf ? pick_norm<true, kResBf16>(p, num_sms, s) : pick_norm<false, kResBf16>(p, num_sms, s);
}

int64_t rmsnorm_bwd_max_blocks(int64_t t) { return t < kNormBwdMaxBlocks ? t : kNormBwdMaxBlocks; }

cudaError_t launch_rmsnorm_bwd(const sbl_rmsnorm_backward_args& a, int num_sms, cudaStream_t s) {
  NormBwdParams p;
  p.h = a.h, p.rstd = a.rstd, p.w = a.weight;
  for (int i = 0; i < 3; ++i) p.dy[i] = i < a.dy_count ? a.dys[i] : nullptr;
  p.ndy = a.dy_count, p.dres = a.dres;
  p.t = a.t, p.nvec = static_cast<int>(a.k / 8);
  p.inv_k = 1.0f / static_cast<float>(a.k);
  p.w_f32 = (a.flags & SBL_NORM_W_F32) != 0u;
  p.dh = a.dh, p.dx = a.dx;
  p.part = a.dw != nullptr ? static_cast<float*>(a.workspace) : nullptr;
  if (num_sms > kNormBwdMaxBlocks) num_sms = kNormBwdMaxBlocks;
  const bool hf = (a.flags & SBL_NORM_STREAM_F32) != 0u, df = (a.flags & SBL_NORM_DY_F32) != 0u;
  if (hf) return df ? pick_norm_bwd<true, true>(p, a.dw, num_sms, s) : pick_norm_bwd<true, false>(p, a.dw, num_sms, s);
  return df ? pick_norm_bwd<false, true>(p, a.dw, num_sms, s) : pick_norm_bwd<false, false>(p, a.dw, num_sms, s);
}

}  // namespace sbl
