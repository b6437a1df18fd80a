// AdamW over many tensors in one launch, states in fp32 or in 8 bits.
//
//   g = grad scale,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   value = value (1 - lr wd) - lr (m / c1) / (sqrt(v / c2) + eps),  c = 1 - b^step
//
// Elementwise: bound by the bytes of the states and weights (28 a weight with
// fp32 states, master and a bf16 gradient; 16 with 8-bit states).  The tensors'
// addresses travel as kernel parameters, so a launch needs no device table and
// can be captured; a block finds its tensor by its chunk's number.
//
// 8-bit states: a warp holds a block of 256 elements, 8 a lane, so the block's
// largest magnitude is one warp reduction.  A value is e4m3 code times scale,
// the second moment through its square root, which halves the exponent range
// it needs.  Nearest rounding, half a step 2^-4 relative; the second moment
// never rounds to zero (the smallest code stands in), since a zero would let
// the next step divide by eps.
//
// Measured, the 79 M weights of a transformer block (four 2560 x 2560, three 6912 x
// 2560, vectors) in one launch: fp32 states 327 us (6.8 TB/s, a little over
// the copy's rate); 8-bit states 205 us (6.2 TB/s; 53 instructions a weight, two
// reductions a block among them).
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "f32x2.cuh"
#include "sbl_device.cuh"
#include "sbl_kernels.h"

namespace sbl {

namespace {

// Blocks of 128 threads: with 8-bit states nine of them have 56 registers a thread
// (79 M weights in a graph 190 us; four blocks of 256 with 64 registers 210, ten of
// 128 with 48 and spills 203).  Elements of one tensor that a block updates: 16 a
// thread with fp32 states (327 -> 324 us against blocks of 256, 90 k weights 5.9 ->
// 3.7; 8 a thread 325 and 5.1), one 8-bit block a warp.
constexpr int kAdamThreads = 128;
constexpr int chunk_of(bool eight) { return eight ? kAdamThreads / 32 * SBL_ADAMW_BLOCK : 16 * kAdamThreads; }
constexpr float kFlush = 0x1p-100f;
constexpr float kFp8Max = 448.0f, kFp8Min = 0x1p-9f;

struct AdamEntry {
  void* w;
  float* master;
  const void* grad;
  void *m, *v;
  float *m_scale, *v_scale;
  int64_t numel;
  uint32_t flags;
};

// The step's scalars.
struct AdamStep {
  float b1, one_b1, b2, one_b2, eps;
  float keep;      // 1 - lr decay
  float rate;      // lr / (1 - b1^step)
  float inv_root;  // 1 / sqrt(1 - b2^step)
  float scale;     // of the gradients
};

struct AdamLaunch {
  AdamEntry entry[kAdamMaxTensors];
  uint32_t first[kAdamMaxTensors + 1];  // first chunk of each tensor
  int count;
  AdamStep step;
  // for the scalars that live on the device
  float lr, decay;
  double log_b1, log_b2, n;
  const float* lr_dev;
  const int64_t* step_dev;
  const float* grad_scale_dev;
  uint32_t* status;
};

__device__ __forceinline__ AdamStep adam_step(const AdamLaunch& p, bool no_decay) {
  AdamStep s = p.step;
  if (p.lr_dev != nullptr || p.step_dev != nullptr) {
    const float lr = p.lr_dev != nullptr ? *p.lr_dev : p.lr;
    const double n = p.step_dev != nullptr ? static_cast<double>(*p.step_dev) : p.n;
    s.keep = 1.0f - lr * p.decay;
    s.rate = lr / static_cast<float>(-expm1(n * p.log_b1));
    s.inv_root = 1.0f / sqrtf(static_cast<float>(-expm1(n * p.log_b2)));
  }
  if (no_decay) s.keep = 1.0f;
  if (p.grad_scale_dev != nullptr) s.scale = *p.grad_scale_dev;
  return s;
}

// One element with fp32 states; m, v and value are updated.  The moments'
// products and sums are rounded one by one (no fused multiply-add): the states are
// then the same on every build and in any plain form.
__device__ __forceinline__ void adam_element(const AdamStep& s, float grad, float& m, float& v, float& value,
                                             uint32_t& bad) {
  const float g = __fmul_rn(grad, s.scale);
  bad = max(bad, __float_as_uint(g) & 0x7FFFFFFFu);
  m = __fadd_rn(__fmul_rn(s.b1, m), __fmul_rn(s.one_b1, g));
  v = __fadd_rn(__fmul_rn(s.b2, v), __fmul_rn(__fmul_rn(s.one_b2, g), g));
  // the quotient is off by two units at most; nothing rounds behind it
  value = fmaf(value, s.keep, -__fdividef(s.rate * m, fmaf(__fsqrt_rn(v), s.inv_root, s.eps)));
}

template <bool F32>
__device__ __forceinline__ void load4(const void* base, int64_t i, float (&f)[4]) {
  if constexpr (F32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
    f[0] = __uint_as_float(a.x << 16), f[1] = __uint_as_float(a.x & 0xFFFF0000u);
    f[2] = __uint_as_float(a.y << 16), f[3] = __uint_as_float(a.y & 0xFFFF0000u);
  }
}

__device__ __forceinline__ float load1(const void* base, int64_t i, bool f32) {
  if (f32) return static_cast<const float*>(base)[i];
  return __uint_as_float(uint32_t(static_cast<const uint16_t*>(base)[i]) << 16);
}

__device__ __forceinline__ void store4(float* base, int64_t i, const float (&f)[4]) {
  *reinterpret_cast<float4*>(base + i) = make_float4(f[0], f[1], f[2], f[3]);
}

__device__ __forceinline__ void store4_bf16(void* base, int64_t i, const float (&f)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// The four e4m3 codes of a word, as two pairs.
__device__ __forceinline__ void from_fp8(uint32_t word, f32x2 (&f)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw raw = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(word >> (16 * h)), __NV_E4M3);
    const float2 v = __half22float2(__half2(raw));
    f[h] = pair(v.x, v.y);
  }
}

__device__ __forceinline__ uint32_t to_fp8(f32x2 a, f32x2 b) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(halves(a), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(halves(b), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

__device__ __forceinline__ float rsqrt_fast(float x) {
  float y;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The sum of two rounded products, by scalar additions (see f32x2.cuh).
__device__ __forceinline__ f32x2 sum_of_products(f32x2 a, f32x2 b) {
  const float2 p = halves(a), q = halves(b);
  return pair(__fadd_rn(p.x, q.x), __fadd_rn(p.y, q.y));
}

// Square roots of two values from 2^-100 up, by Newton's step on g = v y with
// y near 1 / sqrt(v) (Markstein, IBM J. Res. Dev. 1990): r = g + (v - g^2) y / 2,
// the residual exact in a fused multiply-add.  The result before its rounding
// is within 2^-44 (relative), so it is the rounded root but for about one value
// in two million, there its neighbour: a second moment's code differs from that of
// the rounded root only where such a value also lies next to a border of two codes.
__device__ __forceinline__ f32x2 root2(f32x2 v) {
  const float2 f = halves(v);
  const f32x2 y = pair(rsqrt_fast(f.x), rsqrt_fast(f.y));
  const f32x2 g = mul2(v, y), half = mul2(y, pair(0.5f, 0.5f));
  return fma2(fma2(mul2(g, pair(-1.0f, -1.0f)), g, v), half, g);
}

template <bool GF32, bool MASTER>
__device__ __forceinline__ void update_fp32(const AdamEntry& t, const AdamStep& s, int64_t first, uint32_t& bad) {
  constexpr int kChunk = chunk_of(false), U = kChunk / (4 * kAdamThreads);
  float* mp = static_cast<float*>(t.m);
  float* vp = static_cast<float*>(t.v);
  const int64_t at = first + 4 * threadIdx.x;
  if (first + kChunk <= t.numel) {
    float g[U][4], m[U][4], v[U][4], x[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = at + u * 4 * kAdamThreads;
      load4<GF32>(t.grad, i, g[u]);
      load4<true>(mp, i, m[u]);
      load4<true>(vp, i, v[u]);
      load4<MASTER>(MASTER ? static_cast<const void*>(t.master) : t.w, i, x[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = at + u * 4 * kAdamThreads;
#pragma unroll
      for (int e = 0; e < 4; ++e) adam_element(s, g[u][e], m[u][e], v[u][e], x[u][e], bad);
      store4(mp, i, m[u]);
      store4(vp, i, v[u]);
      if (MASTER) store4(t.master, i, x[u]);
      store4_bf16(t.w, i, x[u]);
    }
    return;
  }
  for (int64_t i = first + threadIdx.x; i < t.numel; i += kAdamThreads) {
    float x = MASTER ? t.master[i] : load1(t.w, i, false), m = mp[i], v = vp[i];
    adam_element(s, load1(t.grad, i, GF32), m, v, x, bad);
    mp[i] = m;
    vp[i] = v;
    if (MASTER) t.master[i] = x;
    static_cast<__nv_bfloat16*>(t.w)[i] = __float2bfloat16_rn(x);
  }
}

// Largest magnitude of the warp's values (their bits order as the values do).
__device__ __forceinline__ float warp_top(float top) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
}

// A block of 256 elements by one warp, 8 consecutive ones a lane, in pairs.  Behind
// the moments stands the rounding to 8 bits, where one unit in the last place
// decides between two codes 6 to 12 % apart: so their products and sums are
// rounded one by one here too, and the largest value's root, which gives the scale,
// is the IEEE one.  First moments and both scales are those of any plain form;
// second moments' codes are but for root2's neighbours.
template <bool GF32, bool MASTER>
__device__ __forceinline__ void update_fp8(const AdamEntry& t, const AdamStep& s, int64_t first, uint32_t& bad) {
  const int lane = threadIdx.x & 31;
  const int64_t start = first + (threadIdx.x >> 5) * SBL_ADAMW_BLOCK;
  if (start >= t.numel) return;
  const int64_t block = start / SBL_ADAMW_BLOCK, i = start + 8 * lane;
  uint8_t* mp = static_cast<uint8_t*>(t.m) + i;
  uint8_t* vp = static_cast<uint8_t*>(t.v) + i;
  const bool full = start + SBL_ADAMW_BLOCK <= t.numel;
  float gf[2][4], xf[2][4];
  uint2 mw = make_uint2(0, 0), vw = make_uint2(0, 0);
  const float ms = t.m_scale[block], vs = t.v_scale[block];
  if (full) {
    mw = *reinterpret_cast<const uint2*>(mp);
    vw = *reinterpret_cast<const uint2*>(vp);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load4<GF32>(t.grad, i + 4 * h, gf[h]);
      load4<MASTER>(MASTER ? static_cast<const void*>(t.master) : t.w, i + 4 * h, xf[h]);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t j = i + 4 * h + e;
        const bool in = j < t.numel;
        gf[h][e] = in ? load1(t.grad, j, GF32) : 0.0f;
        xf[h][e] = in ? (MASTER ? t.master[j] : load1(t.w, j, false)) : 0.0f;
        (h ? mw.y : mw.x) |= in ? uint32_t(mp[4 * h + e]) << (8 * e) : 0u;
        (h ? vw.y : vw.x) |= in ? uint32_t(vp[4 * h + e]) << (8 * e) : 0u;
      }
  }
  f32x2 m[4], v[4];
  {
    f32x2 a[2], b[2];
    from_fp8(mw.x, a);
    from_fp8(mw.y, b);
    m[0] = a[0], m[1] = a[1], m[2] = b[0], m[3] = b[1];
    from_fp8(vw.x, a);
    from_fp8(vw.y, b);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
  }
  float mtop = 0.0f;
  uint32_t vtop = 0, vlow = 0x7F800000u;  // the second moments' bits, which order as they do
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const f32x2 g = mul2(pair(gf[e >> 1][2 * (e & 1)], gf[e >> 1][2 * (e & 1) + 1]), pair(s.scale, s.scale));
    m[e] = sum_of_products(mul2(pair(s.b1, s.b1), mul2(m[e], pair(ms, ms))), mul2(pair(s.one_b1, s.one_b1), g));
    v[e] = mul2(v[e], pair(vs, vs));
    v[e] = sum_of_products(mul2(pair(s.b2, s.b2), mul2(v[e], v[e])), mul2(mul2(pair(s.one_b2, s.one_b2), g), g));
    const float2 a = halves(m[e]), b = halves(v[e]);
    mtop = fmaxf(mtop, fmaxf(fabsf(a.x), fabsf(a.y)));
    const uint32_t b0 = __float_as_uint(b.x), b1 = __float_as_uint(b.y);
    vtop = max(vtop, max(b0, b1));
    vlow = min(vlow, min(b0, b1));
  }
  mtop = warp_top(mtop);
  vtop = __reduce_max_sync(0xffffffffu, vtop);
  bad = max(bad, vtop);
  const float rtop = __fsqrt_rn(__uint_as_float(vtop));
  // pinned like the moments: 448 times the reciprocal, and the top times 1 / 448
  const float mi = mtop >= kFlush ? __fmul_rn(kFp8Max, __frcp_rn(mtop)) : 0.0f;
  const float vi = rtop >= kFlush ? __fmul_rn(kFp8Max, __frcp_rn(rtop)) : 0.0f;
  if (lane == 0) {
    t.m_scale[block] = mtop >= kFlush ? __fmul_rn(mtop, 1.0f / kFp8Max) : 0.0f;
    t.v_scale[block] = rtop >= kFlush ? __fmul_rn(rtop, 1.0f / kFp8Max) : 0.0f;
  }
  // Where no root is below a smallest code (448 2^-9 of the top: 2^-36 of the
  // top's square, with room) nor outside root2's range, none needs a look.
  f32x2 r[4];
  const float low = __uint_as_float(vlow);
  const bool plain = low >= 0x1p-100f && low >= 0x1p-34f * __uint_as_float(vtop);
  if (__all_sync(0xffffffffu, plain)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r[e] = root2(v[e]);
      v[e] = mul2(r[e], pair(vi, vi));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = halves(v[e]), b = make_float2(__fsqrt_rn(a.x), __fsqrt_rn(a.y));
      r[e] = pair(b.x, b.y);
      float q0 = __fmul_rn(b.x, vi), q1 = __fmul_rn(b.y, vi);
      if (q0 > 0.0f) q0 = fmaxf(q0, kFp8Min);
      if (q1 > 0.0f) q1 = fmaxf(q1, kFp8Min);
      v[e] = pair(q0, q1);
    }
  }
  f32x2 x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 den = halves(fma2(r[e], pair(s.inv_root, s.inv_root), pair(s.eps, s.eps)));
    const float2 num = halves(mul2(m[e], pair(-s.rate, -s.rate)));
    // the quotients are off by two units at most; nothing rounds behind them
    x[e] = fma2(pair(xf[e >> 1][2 * (e & 1)], xf[e >> 1][2 * (e & 1) + 1]), pair(s.keep, s.keep),
                pair(__fdividef(num.x, den.x), __fdividef(num.y, den.y)));
    m[e] = mul2(m[e], pair(mi, mi));
  }
  mw = make_uint2(to_fp8(m[0], m[1]), to_fp8(m[2], m[3]));
  vw = make_uint2(to_fp8(v[0], v[1]), to_fp8(v[2], v[3]));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = halves(x[e]);
    xf[e >> 1][2 * (e & 1)] = a.x;
    xf[e >> 1][2 * (e & 1) + 1] = a.y;
  }
  if (full) {
    *reinterpret_cast<uint2*>(mp) = mw;
    *reinterpret_cast<uint2*>(vp) = vw;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (MASTER) store4(t.master, i + 4 * h, xf[h]);
      store4_bf16(t.w, i + 4 * h, xf[h]);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t j = i + 4 * h + e;
        if (j >= t.numel) continue;
        mp[4 * h + e] = static_cast<uint8_t>((h ? mw.y : mw.x) >> (8 * e));
        vp[4 * h + e] = static_cast<uint8_t>((h ? vw.y : vw.x) >> (8 * e));
        if (MASTER) t.master[j] = xf[h][e];
        static_cast<__nv_bfloat16*>(t.w)[j] = __float2bfloat16_rn(xf[h][e]);
      }
  }
}

template <bool EIGHT>
__global__ void __launch_bounds__(kAdamThreads, EIGHT ? 9 : 4) k_adamw(const __grid_constant__ AdamLaunch p) {
  int lo = 0, hi = p.count - 1;  // the last tensor whose first chunk is not past this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.first[mid] <= blockIdx.x)
      lo = mid;
    else
      hi = mid - 1;
  }
  const AdamEntry t = p.entry[lo];
  const int64_t first = int64_t(blockIdx.x - p.first[lo]) * chunk_of(EIGHT);
  pdl_wait();
  pdl_trigger();
  const AdamStep s = adam_step(p, (t.flags & SBL_ADAMW_NO_DECAY) != 0u);
  uint32_t bad = 0;
  const bool gf = (t.flags & SBL_ADAMW_GRAD_F32) != 0u, master = t.master != nullptr;
  if constexpr (EIGHT) {
    if (gf)
      master ? update_fp8<true, true>(t, s, first, bad) : update_fp8<true, false>(t, s, first, bad);
    else
      master ? update_fp8<false, true>(t, s, first, bad) : update_fp8<false, false>(t, s, first, bad);
  } else {
    if (gf)
      master ? update_fp32<true, true>(t, s, first, bad) : update_fp32<true, false>(t, s, first, bad);
    else
      master ? update_fp32<false, true>(t, s, first, bad) : update_fp32<false, false>(t, s, first, bad);
  }
  if (bad >= 0x7F800000u) raise_status(p.status, SBL_STATUS_NONFINITE_G);
}

}  // namespace

// The tensors of a launch all hold their states alike (the first one's way).
cudaError_t launch_adamw(const sbl_adamw_tensor* tensors, int count, const sbl_adamw_params& q, uint32_t* status,
                         cudaStream_t s) {
  if (count < 1 || count > kAdamMaxTensors) return cudaErrorInvalidValue;
  const bool eight = (tensors[0].flags & SBL_ADAMW_STATE_8BIT) != 0u;
  const uint64_t chunk = static_cast<uint64_t>(chunk_of(eight));
  AdamLaunch p;  // entries and first chunks past `count` are not read
  uint64_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    const sbl_adamw_tensor& t = tensors[i];
    p.entry[i] = AdamEntry{t.w, t.master, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.numel, t.flags};
    p.first[i] = static_cast<uint32_t>(chunks);
    chunks += (uint64_t(t.numel) + chunk - 1) / chunk;
    if (chunks > 0x7FFFFFFFull) return cudaErrorInvalidValue;
  }
  p.first[count] = static_cast<uint32_t>(chunks);
  p.count = count;
  p.lr = static_cast<float>(q.lr), p.decay = static_cast<float>(q.weight_decay);
  p.n = static_cast<double>(q.step), p.log_b1 = std::log(q.beta1), p.log_b2 = std::log(q.beta2);
  p.step.b1 = static_cast<float>(q.beta1), p.step.one_b1 = static_cast<float>(1.0 - q.beta1);
  p.step.b2 = static_cast<float>(q.beta2), p.step.one_b2 = static_cast<float>(1.0 - q.beta2);
  p.step.eps = static_cast<float>(q.eps);
  p.step.keep = static_cast<float>(1.0 - q.lr * q.weight_decay);
  p.step.rate = static_cast<float>(q.lr / -std::expm1(p.n * p.log_b1));
  p.step.inv_root = static_cast<float>(1.0 / std::sqrt(-std::expm1(p.n * p.log_b2)));
  p.step.scale = 1.0f;
  p.lr_dev = q.lr_dev, p.step_dev = q.step_dev, p.grad_scale_dev = q.grad_scale_dev;
  p.status = status;
  return launch_pdl(eight ? k_adamw<true> : k_adamw<false>, dim3(static_cast<unsigned>(chunks)), dim3(kAdamThreads), 0,
                    s, p);
}

}  // namespace sbl
