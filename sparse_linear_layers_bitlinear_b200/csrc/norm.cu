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
#include <algorithm>

#include <cuda_bf16.h>

#include "actq_math.cuh"
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

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t vec, const float (&f)[8]) {
  if constexpr (F32) {
    float4* dst = static_cast<float4*>(base) + 2 * vec;
    dst[0] = make_float4(f[0], f[1], f[2], f[3]);
    dst[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    static_cast<uint4*>(base)[vec] = pack8(f);
  }
}

// RN_fp32(1 / sqrt(a)): the fp32 reciprocal root and two Newton steps in fp64
// (relative error far below fp64's 2^-53 of the exact step), one rounding.
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

// Two fp32 values in a register pair: sm_100's packed fp32 instructions, each
// half rounded as the scalar ones do.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 halves(f32x2 v) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
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
__global__ void __launch_bounds__(ONE_WARP ? 128 : FEW || RES == kNoRes ? kNormMaxWarps * 32 : kNormRowWarps * 32, 1) k_rmsnorm(const NormParams p) {
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
    if (smem > 48 * 1024)
      e = cudaFuncSetAttribute(k_rmsnorm<XF32, RES, R, ONE_WARP, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(smem));
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
// A group of threads walks rows with a fixed stride and keeps its columns'
// share of dw in registers; the groups of a block add theirs in shared memory
// in a fixed order, one row of partial sums a block goes to the workspace,
// and a second launch adds those, in a fixed order too.
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
  void* dh;
  uint4* dx;
  float* part;  // [gridDim.x][k], or nullptr without dw
};

constexpr int kNormBwdBlock(int tpr) { return tpr < 128 ? 256 : 512; }

// The row's threads wait for each other (its own barrier for each group).
template <int TPR>
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
}

template <bool HF32, bool DF32, int TPR, int R>
__global__ void __launch_bounds__(kNormBwdBlock(TPR), 1) k_rmsnorm_bwd(const NormBwdParams p) {
  constexpr int kBlock = kNormBwdBlock(TPR), kGroups = kBlock / TPR, kWarps = TPR / 32;
  __shared__ float s_part[2][kGroups][kWarps];
  __shared__ float4 s_dw[kGroups > 1 ? TPR * R * 2 : 1];
  pdl_wait();
  pdl_trigger();
  const int group = threadIdx.x / TPR, tid = threadIdx.x % TPR, lane = threadIdx.x & 31, warp = tid >> 5;
  float acc[R][8];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[r][e] = 0.0f;

  int parity = 0;
  for (int64_t row = int64_t(blockIdx.x) * kGroups + group; row < p.t; row += int64_t(gridDim.x) * kGroups) {
    const int64_t base = row * p.nvec;
    const float rstd = p.rstd[row];
    float n[R][8], g[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = r * TPR + tid;
#pragma unroll
      for (int e = 0; e < 8; ++e) n[r][e] = g[r][e] = 0.0f;
      if (i < p.nvec) {
        load8<HF32>(p.h, base + i, n[r]);
        load8<DF32>(p.dy[0], base + i, g[r]);
        float q[8];
        if (p.ndy > 1) {
          load8<DF32>(p.dy[1], base + i, q);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[r][e] += q[e];
        }
        if (p.ndy > 2) {
          load8<DF32>(p.dy[2], base + i, q);
#pragma unroll
          for (int e = 0; e < 8; ++e) g[r][e] += q[e];
        }
      }
    }
    float c = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = r * TPR + tid;
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.0f;
      if (p.w != nullptr && i < p.nvec) {
        if (p.w_f32)
          load8<true>(p.w, i, w);
        else
          load8<false>(p.w, i, w);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[r][e] *= rstd;
        acc[r][e] = fmaf(g[r][e], n[r][e], acc[r][e]);
        g[r][e] *= w[e];
        c = fmaf(g[r][e], n[r][e], c);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if constexpr (TPR > 32) {
      if (lane == 0) s_part[parity][group][warp] = c;
      group_sync<TPR>(group);
      c = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) c += s_part[parity][group][i];
      parity ^= 1;  // a slot is written again two rows on, behind another barrier
    }
    c *= p.inv_k;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = r * TPR + tid;
      if (i >= p.nvec) continue;
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = rstd * fmaf(-n[r][e], c, g[r][e]);
      if (p.dres != nullptr) {
        float q[8];
        load8<HF32>(p.dres, base + i, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] += q[e];
      }
      store8<HF32>(p.dh, base + i, d);
      if (p.dx != nullptr) p.dx[base + i] = pack8(d);
    }
  }
  if (p.part == nullptr) return;
  float4* dst = reinterpret_cast<float4*>(p.part) + int64_t(blockIdx.x) * (2 * p.nvec);
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = r * TPR + tid;
      if (i >= p.nvec) continue;
      dst[2 * i] = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
      dst[2 * i + 1] = make_float4(acc[r][4], acc[r][5], acc[r][6], acc[r][7]);
    }
  } else {  // the groups' shares, one group after the other
    for (int gr = 0; gr < kGroups; ++gr) {
      if (group == gr) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float4* s = s_dw + 2 * (r * TPR + tid);
          float4 a = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
          float4 b = make_float4(acc[r][4], acc[r][5], acc[r][6], acc[r][7]);
          if (gr > 0) {
            a.x += s[0].x, a.y += s[0].y, a.z += s[0].z, a.w += s[0].w;
            b.x += s[1].x, b.y += s[1].y, b.z += s[1].z, b.w += s[1].w;
          }
          s[0] = a, s[1] = b;
        }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < 2 * p.nvec; i += kBlock) dst[i] = s_dw[i];
  }
}

// dw[c] = sum of the blocks' partial sums: 8 threads of 4 columns across, 32 rows of
// partial sums at a time, then a tree over the 32.
__global__ void __launch_bounds__(256) k_norm_dw(const float4* __restrict__ part, int blocks, int n4, float4* dw) {
  __shared__ float4 s[32][8];
  pdl_wait();
  pdl_trigger();
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int col = blockIdx.x * 8 + x;
  float4 a = make_float4(0, 0, 0, 0);
  if (col < n4)
    for (int b = y; b < blocks; b += 32) {
      const float4 v = __ldcg(part + int64_t(b) * n4 + col);
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
  s[y][x] = a;
  for (int o = 16; o > 0; o >>= 1) {
    __syncthreads();
    if (y < o) {
      const float4 v = s[y + o][x];
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
      s[y][x] = a;
    }
  }
  if (y == 0 && col < n4) dw[col] = a;
}

template <bool HF32, bool DF32, int TPR, int R>
cudaError_t launch_norm_bwd(NormBwdParams p, float* dw, int num_sms, cudaStream_t s) {
  constexpr int block = kNormBwdBlock(TPR), groups = block / TPR;
  const int64_t want = (p.t + groups - 1) / groups;
  const int blocks = static_cast<int>(want < num_sms ? want : num_sms);
  const cudaError_t e =
      launch_pdl(k_rmsnorm_bwd<HF32, DF32, TPR, R>, dim3(blocks), dim3(block), 0, s, p);
  if (e != cudaSuccess || dw == nullptr) return e;
  const int n4 = 2 * p.nvec;
  return launch_pdl(k_norm_dw, dim3((n4 + 7) / 8), dim3(256), 0, s, reinterpret_cast<const float4*>(p.part), blocks,
                    n4, reinterpret_cast<float4*>(dw));
}

template <bool HF32, bool DF32>
cudaError_t pick_norm_bwd(const NormBwdParams& p, float* dw, int num_sms, cudaStream_t s) {
  const int n = p.nvec;
  if (n <= 32) return launch_norm_bwd<HF32, DF32, 32, 1>(p, dw, num_sms, s);
  if (n <= 64) return launch_norm_bwd<HF32, DF32, 32, 2>(p, dw, num_sms, s);
  if (n <= 128) return launch_norm_bwd<HF32, DF32, 32, 4>(p, dw, num_sms, s);
  if (n <= 256) return launch_norm_bwd<HF32, DF32, 128, 2>(p, dw, num_sms, s);
  if (n <= 384) return launch_norm_bwd<HF32, DF32, 128, 3>(p, dw, num_sms, s);
  if (n <= 512) return launch_norm_bwd<HF32, DF32, 128, 4>(p, dw, num_sms, s);
  if (n <= 1024) return launch_norm_bwd<HF32, DF32, 512, 2>(p, dw, num_sms, s);
  if (n <= 1536) return launch_norm_bwd<HF32, DF32, 512, 3>(p, dw, num_sms, s);
  return launch_norm_bwd<HF32, DF32, 512, 4>(p, dw, num_sms, s);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, int num_sms, cudaStream_t s) {
  NormParams p;
  p.x = a.x, p.res = a.residual, p.w = a.weight;
  p.t = a.t, p.nvec = static_cast<int>(a.k / 8);
  p.inv_k = 1.0 / static_cast<double>(a.k), p.eps = a.eps;
  p.w_f32 = (a.flags & SBL_NORM_W_F32) != 0u;
  p.h = a.h;
  p.xn = static_cast<uint4*>(a.xn), p.xhat = static_cast<uint4*>(a.xhat), p.xq = reinterpret_cast<uint2*>(a.xq);
  p.xscale = a.xscale, p.rstd = a.rstd, p.status = a.status;
  const bool xf = (a.flags & SBL_NORM_X_F32) != 0u, rf = (a.flags & SBL_NORM_STREAM_F32) != 0u;
  if (a.residual == nullptr) return xf ? pick_norm<true, kNoRes>(p, num_sms, s) : pick_norm<false, kNoRes>(p, num_sms, s);
  if (rf) return xf ? pick_norm<true, kResF32>(p, num_sms, s) : pick_norm<false, kResF32>(p, num_sms, s);
  return xf ? pick_norm<true, kResBf16>(p, num_sms, s) : pick_norm<false, kResBf16>(p, num_sms, s);
}

int64_t rmsnorm_bwd_max_blocks(int64_t t) { return t < kNormBwdMaxBlocks ? t : kNormBwdMaxBlocks; }

cudaError_t launch_rmsnorm_bwd(const NormBwdArgs& a, int num_sms, cudaStream_t s) {
  NormBwdParams p;
  p.h = a.h, p.rstd = a.rstd, p.w = a.weight;
  for (int i = 0; i < 3; ++i) p.dy[i] = i < a.dy_count ? a.dys[i] : nullptr;
  p.ndy = a.dy_count, p.dres = a.dres;
  p.t = a.t, p.nvec = static_cast<int>(a.k / 8);
  p.inv_k = 1.0f / static_cast<float>(a.k);
  p.w_f32 = (a.flags & SBL_NORM_W_F32) != 0u;
  p.dh = a.dh, p.dx = static_cast<uint4*>(a.dx);
  p.part = a.dw != nullptr ? static_cast<float*>(a.workspace) : nullptr;
  if (num_sms > kNormBwdMaxBlocks) num_sms = kNormBwdMaxBlocks;
  const bool hf = (a.flags & SBL_NORM_STREAM_F32) != 0u, df = (a.flags & SBL_NORM_DY_F32) != 0u;
  if (hf) return df ? pick_norm_bwd<true, true>(p, a.dw, num_sms, s) : pick_norm_bwd<true, false>(p, a.dw, num_sms, s);
  return df ? pick_norm_bwd<false, true>(p, a.dw, num_sms, s) : pick_norm_bwd<false, false>(p, a.dw, num_sms, s);
}

}  // namespace sbl
