// Softmax cross entropy of a linear head without its logits in memory, on the
// CTA-pair tensor-core GEMM (gemm_pair.cuh).
//
//   z = h w^T,  lse_i = log sum_j exp z_ij,  loss_i = lse_i - z_i,target_i
//   dz_ij = dloss_i (exp(z_ij - lse_i) - [j = target_i]),  dh = dz w,  dw = dz^T h
//
// Forward: a tile of 256 tokens x 256 vocabulary entries leaves, per token, its
// largest logit and the sum of the exponentials below it (the epilogue's eight
// warps keep a half tile each); a second launch joins a token's pieces.  The
// product bounds it: 2 t v d flops; the exponentials (one per logit) run on
// the epilogue warps under the next tile's product.
//
// Backward, a piece of the vocabulary at a time, so that dz (bf16, at most
// kCeDzBytes) stays in L2 between its writer and its two readers: one launch
// computes the piece's logits again and writes dz, a second one runs both
// products over it.  dw rows belong to one piece; dh adds up over the pieces
// in fp32.  With few tokens dh has few output tiles and a long sum over the
// vocabulary, which is then split over slices that a last launch joins.
#include <algorithm>

#include "gemm_launch.cuh"

namespace sbl {

namespace {

constexpr int kCeTile = 256;

__device__ __forceinline__ float exp_of(float x) {  // exp(x), x <= 0 or slightly above
  return exp2f(x * 1.4426950408889634f);
}

// Common form of the h . w^T tiles: A = h rows, B = w rows, both K-major.
template <class P>
struct CfgCeLogits {
  using Params = P;
  static constexpr bool QUANT_X = false;
  static constexpr int MAPS = 2;
  static constexpr int EPI_WARPS = 8;
  static constexpr int BN = kCeTile, BK = 64, STAGES = 6;
  static constexpr int A_BYTES = 128 * BK * 2;       // 16 KB
  static constexpr int B_BYTES = (BN / 2) * BK * 2;  // 16 KB
  static constexpr int E_BYTES = 0;
  static constexpr int ACC_COLS = BN;
  static constexpr int TMEM_COLS = 512;
  static constexpr int E_COL0 = 0, E_COLS = 0;
  static constexpr uint32_t IDESC = idesc_bf16(256, BN, false, false);

  __device__ static int rows_M(const P& p) { return p.t; }
  __device__ static int cols_N(const P& p) { return p.v; }
  __device__ static int k_blocks(const P& p) { return (p.d + BK - 1) / BK; }

  __device__ static void load_stage(const CUtensorMap* tA, const CUtensorMap* tB, const CUtensorMap*,
                                    const CUtensorMap*, const P&, int, uint8_t* sA, uint8_t* sB, uint8_t*, int m0,
                                    int n0, int kb, uint64_t* bar) {
    tma_load_2d_pair(sA, tA, kb * BK, m0, bar);
    tma_load_2d_pair(sB, tB, kb * BK, n0, bar);
  }

  __device__ static void mma_stage(const P&, int, uint32_t d_tmem, uint32_t, uint8_t* sA, uint8_t* sB, uint8_t*,
                                   bool first) {
    const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB);
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk)
      mma_bf16_pair(d_tmem, smem_desc(a0 + kk * 32, 16, 1024, 2), smem_desc(b0 + kk * 32, 16, 1024, 2), IDESC,
                    (first && kk == 0) ? 0u : 1u);
  }
};

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
struct CeFwdParams {
  int t, v, d;
  int pieces;     // per token: two for each vocabulary tile
  float2* piece;  // [t][pieces]: largest logit, sum of exp(logit - largest)
  float* hit;     // [t]: the target's logit
  const int64_t* targets;
  uint32_t* status;
};

struct CfgCeFwd : CfgCeLogits<CeFwdParams> {
  using Tiles = StripedTiles<CfgCeFwd>;

  __device__ static void epilogue(const CeFwdParams& p, int, uint32_t t_acc, int row, int n0, int, int part,
                                  int parts) {
    const bool in = row < p.t;
    const int64_t target = in ? __ldcg(p.targets + row) : -1;
    float top = -INFINITY, sum = 0.0f;
#pragma unroll 1
    for (int c = part; c < BN / 32; c += parts) {
      const int col0 = n0 + c * 32;
      if (col0 >= p.v) break;  // uniform across the warp
      uint32_t r[32];
      __syncwarp();
      tmem_load_32x32b_x32(t_acc + c * 32, r);
      tmem_load_wait();
      const int left = p.v - col0;
      float z[32], best = top;
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        z[e] = e < left ? __uint_as_float(r[e]) : -INFINITY;
        best = fmaxf(best, z[e]);
      }
      const int64_t at = target - col0;
      if (at >= 0 && at < 32 && in) {
        float hit = 0.0f;
#pragma unroll
        for (int e = 0; e < 32; ++e) hit = e == int(at) ? z[e] : hit;
        if (target < p.v) p.hit[row] = hit;
      }
      const float base = best == -INFINITY ? 0.0f : best;
      sum *= exp_of(top - base);
#pragma unroll
      for (int e = 0; e < 32; ++e) sum += exp_of(z[e] - base);
      top = best;
    }
    if (in) p.piece[int64_t(row) * p.pieces + 2 * (n0 / BN) + part] = make_float2(top, sum);
  }
};

// One warp a token: the pieces' joint largest logit, then their sum.
__global__ void __launch_bounds__(256)
    k_ce_join(const float2* __restrict__ piece, int pieces, const float* __restrict__ hit,
              const int64_t* __restrict__ targets, int t, int64_t v, int64_t ignore, float* loss, float* lse,
              uint32_t* status) {
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= t) return;
  const float2* src = piece + int64_t(row) * pieces;
  float top = -INFINITY, sum = 0.0f;
  for (int i = lane; i < pieces; i += 32) {
    const float2 q = __ldcg(src + i);
    const float best = fmaxf(top, q.x), base = best == -INFINITY ? 0.0f : best;
    sum = sum * exp_of(top - base) + q.y * exp_of(q.x - base);
    top = best;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float qx = __shfl_xor_sync(0xffffffffu, top, o), qy = __shfl_xor_sync(0xffffffffu, sum, o);
    const float best = fmaxf(top, qx), base = best == -INFINITY ? 0.0f : best;
    sum = sum * exp_of(top - base) + qy * exp_of(qx - base);
    top = best;
  }
  if (lane == 0) {
    const float log_sum = logf(sum);
    const int64_t target = __ldcg(targets + row);
    lse[row] = top + log_sum;
    float l = 0.0f;
    if (target != ignore) {
      if (target >= 0 && target < v) {
        l = (top - __ldcg(hit + row)) + log_sum;
      } else {
        l = __int_as_float(0x7FC00000);
        raise_status(status, SBL_STATUS_BAD_TARGET);
      }
    }
    loss[row] = l;
  }
}

// ---------------------------------------------------------------------------
// Backward: dz of one piece of the vocabulary
// ---------------------------------------------------------------------------
struct CeDzParams {
  int t, v, d;  // v: entries of this piece
  int64_t first;
  int64_t ld;   // elements of a dz row
  uint16_t* dz;
  const int64_t* targets;
  int64_t v_all, ignore;
  const float* lse;
  const float* dloss;
  int64_t dloss_stride;
  uint32_t* status;
};

struct CfgCeDz : CfgCeLogits<CeDzParams> {
  using Tiles = StripedTiles<CfgCeDz>;

  __device__ static void epilogue(const CeDzParams& p, int, uint32_t t_acc, int row, int n0, int, int part,
                                  int parts) {
    const bool in = row < p.t;
    const int64_t target = in ? __ldcg(p.targets + row) : -1;
    const bool good = target >= 0 && target < p.v_all && target != p.ignore;
    if (in && !good && target != p.ignore && n0 == 0 && p.first == 0 && part == 0)
      raise_status(p.status, SBL_STATUS_BAD_TARGET);
    const float lse = in ? __ldcg(p.lse + row) : 0.0f;
    const float scale = good ? __ldcg(p.dloss + row * p.dloss_stride) : 0.0f;
#pragma unroll 1
    for (int c = part; c < BN / 32; c += parts) {
      const int col0 = n0 + c * 32;
      if (col0 >= p.v) break;  // uniform across the warp
      uint32_t r[32];
      __syncwarp();
      tmem_load_32x32b_x32(t_acc + c * 32, r);
      tmem_load_wait();
      if (!in) continue;  // after the warp-wide load
      const int64_t at = target - p.first - col0;
      uint4* dst = reinterpret_cast<uint4*>(p.dz + int64_t(row) * p.ld + col0);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t packed[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y[2];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int j = 8 * q + 2 * e + f;
            float x = exp_of(__uint_as_float(r[j]) - lse);
            if (at == j) x -= 1.0f;
            y[f] = scale != 0.0f ? x * scale : 0.0f;
          }
          const __nv_bfloat162 h2 = __floats2bfloat162_rn(y[0], y[1]);
          packed[e] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        if (col0 + 8 * q < p.v) dst[q] = make_uint4(packed[0], packed[1], packed[2], packed[3]);
      }
    }
  }
};

// ---------------------------------------------------------------------------
// Backward: both products over a piece's dz in one launch.
//   problem 0 (dh):  A = dz [t][v] K-major, B = w piece [v][d] MN-major, K = v
//                    in `slices` runs of k_run blocks of 64
//   problem 1 (dw):  A = dz MN-major (M = v), B = h [t][d] MN-major, K = t
// Tiles of the deeper problem first, striped over the pairs.  A tile's problem
// number carries its slice: 2 * slice for dh, 1 for dw.
// ---------------------------------------------------------------------------
struct CeProductParams {
  int t, v, d;
  int slices, k_run;  // dh: runs of the sum over v
  int mb0, mb1, nb;   // 256-wide blocks of t, v and d
  int dh_first;
  float* acc;         // [slices][t][d] fp32, or nullptr: dh is written directly
  int add;            // acc holds the earlier pieces' sum
  int last;           // with one slice: write dh instead of acc
  uint16_t *dh, *dw;  // dw: this piece's rows
  uint32_t* status;
};

struct CfgCeProducts {
  using Params = CeProductParams;
  static constexpr bool QUANT_X = false;
  static constexpr int MAPS = 4;
  static constexpr int EPI_WARPS = 4;
  static constexpr int BN = kCeTile, BK = 64, STAGES = 6;
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int B_BYTES = (BN / 2) * BK * 2;
  static constexpr int E_BYTES = 0;
  static constexpr int ACC_COLS = BN;
  static constexpr int TMEM_COLS = 512;
  static constexpr int E_COL0 = 0, E_COLS = 0;
  static constexpr uint32_t IDESC0 = idesc_bf16(256, BN, false, true);
  static constexpr uint32_t IDESC1 = idesc_bf16(256, BN, true, true);

  __host__ __device__ static int tiles0(const Params& p) { return p.mb0 * p.nb * p.slices; }
  __host__ __device__ static int tiles1(const Params& p) { return p.mb1 * p.nb; }

  struct Tiles {
    __device__ static int count(const Params& p, int pair, int npairs) {
      const int n = tiles0(p) + tiles1(p);
      return pair < n ? (n - pair + npairs - 1) / npairs : 0;
    }
    __device__ static PairTile at(const Params& p, int pair, int npairs, int i) {
      int id = pair + i * npairs;
      const int first = p.dh_first ? tiles0(p) : tiles1(p);
      const bool dh = (id < first) == (p.dh_first != 0);
      if (id >= first) id -= first;
      if (!dh) return PairTile{1, id % p.mb1, id / p.mb1, (p.t + BK - 1) / BK};
      const int slice = id / (p.mb0 * p.nb);
      id -= slice * p.mb0 * p.nb;
      const int blocks = (p.v + BK - 1) / BK - slice * p.k_run;
      return PairTile{2 * slice, id % p.mb0, id / p.mb0, min(blocks, p.k_run)};
    }
  };

  // Maps: dz (K-major boxes), w, dz (MN-major boxes), h.
  __device__ static void load_stage(const CUtensorMap* tA, const CUtensorMap* tB, const CUtensorMap* tA1,
                                    const CUtensorMap* tB1, const Params& p, int prob, uint8_t* sA, uint8_t* sB,
                                    uint8_t*, int m0, int n0, int kb, uint64_t* bar) {
    if (prob != 1) {
      const int k0 = ((prob >> 1) * p.k_run + kb) * BK;
      tma_load_2d_pair(sA, tA, k0, m0, bar);  // [128 m][64 k]
      tma_load_2d_pair(sB, tB, n0, k0, bar);  // [64 k][64 n] x 2
      tma_load_2d_pair(sB + 8192, tB, n0 + 64, k0, bar);
    } else {
      const int k0 = kb * BK;
      tma_load_2d_pair(sA, tA1, m0, k0, bar);  // [64 k][64 m] x 2
      tma_load_2d_pair(sA + 8192, tA1, m0 + 64, k0, bar);
      tma_load_2d_pair(sB, tB1, n0, k0, bar);
      tma_load_2d_pair(sB + 8192, tB1, n0 + 64, k0, bar);
    }
  }

  __device__ static void mma_stage(const Params&, int prob, uint32_t d_tmem, uint32_t, uint8_t* sA, uint8_t* sB,
                                   uint8_t*, bool first) {
    const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB);
    const bool dw = prob == 1;
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk) {
      const uint64_t ad = dw ? smem_desc(a0 + kk * 2048, 8192, 1024, 2) : smem_desc(a0 + kk * 32, 16, 1024, 2);
      const uint64_t bd = smem_desc(b0 + kk * 2048, 8192, 1024, 2);
      mma_bf16_pair(d_tmem, ad, bd, dw ? IDESC1 : IDESC0, (first && kk == 0) ? 0u : 1u);
    }
  }

  __device__ static void epilogue(const Params& p, int prob, uint32_t t_acc, int row, int n0, int, int part,
                                  int parts) {
    const bool dw = prob == 1;
    const bool to_acc = !dw && p.acc != nullptr && !p.last;
    const bool add = !dw && p.acc != nullptr && p.add;
    const int rows = dw ? p.v : p.t;
    float* acc = to_acc || add ? p.acc + (int64_t(prob >> 1) * p.t + row) * p.d : nullptr;
    uint16_t* out = (dw ? p.dw : p.dh) + int64_t(row) * p.d;
#pragma unroll 1
    for (int c = part; c < BN / 32; c += parts) {
      uint32_t r[32];
      __syncwarp();
      tmem_load_32x32b_x32(t_acc + c * 32, r);
      tmem_load_wait();
      const int col0 = n0 + c * 32;
      if (row >= rows || col0 >= p.d) continue;  // after the warp-wide load
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = col0 + 8 * q;
        if (col >= p.d) break;  // d is a multiple of 8
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(r[8 * q + e]);
        if (add) {  // through L2: another SM may have written it in the launch before
          const float4 a = __ldcg(reinterpret_cast<const float4*>(acc + col));
          const float4 b = __ldcg(reinterpret_cast<const float4*>(acc + col) + 1);
          f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w;
          f[4] += b.x, f[5] += b.y, f[6] += b.z, f[7] += b.w;
        }
        if (to_acc) {
          reinterpret_cast<float4*>(acc + col)[0] = make_float4(f[0], f[1], f[2], f[3]);
          reinterpret_cast<float4*>(acc + col)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
          uint32_t packed[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
            packed[e] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          *reinterpret_cast<uint4*>(out + col) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
        }
      }
    }
  }
};

// dh = the sum of its slices, in their order.
__global__ void __launch_bounds__(256)
    k_ce_dh(const float4* __restrict__ acc, int slices, int64_t n4, uint2* __restrict__ dh) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n4) return;
  float4 a = __ldcg(acc + i);
  for (int s = 1; s < slices; ++s) {
    const float4 b = __ldcg(acc + s * n4 + i);
    a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(a.z, a.w);
  dh[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// How the backward pass cuts its work.
constexpr int64_t kCeDzBytes = int64_t(64) << 20;  // dz of one piece: half of L2

struct CePlan {
  int64_t piece;    // vocabulary entries of a piece, a multiple of 256
  int64_t pieces;
  int slices, k_run;
  uint64_t dz_bytes, acc_bytes;
};

CePlan ce_plan(int64_t t, int64_t v, int64_t d) {
  CePlan c;
  const int64_t padded = (v + 255) / 256 * 256;
  const int64_t most = std::max<int64_t>(kCeDzBytes / (2 * t) / 256, 1) * 256;
  c.pieces = (padded + most - 1) / most;
  c.piece = ((padded / 256 + c.pieces - 1) / c.pieces) * 256;  // even pieces
  c.pieces = (padded + c.piece - 1) / c.piece;
  c.dz_bytes = align_up(uint64_t(t) * uint64_t(c.piece) * 2, 256);
  // dh in one piece's launch: its tiles are as deep as the piece is wide.  A
  // run of the sum is at most what each pair has to do anyway (or 8 blocks).
  const int64_t nb = (d + 255) / 256, mb0 = (t + 255) / 256, mb1 = c.piece / 256;
  const int64_t kb0 = (std::min(c.piece, v) + 63) / 64, kb1 = (t + 63) / 64, pairs = 74;  // 148 SMs
  const int64_t share = std::max<int64_t>((mb0 * nb * kb0 + mb1 * nb * kb1) / pairs, 8);
  int64_t slices = std::min<int64_t>((kb0 + share - 1) / share, 32);
  c.k_run = static_cast<int>((kb0 + slices - 1) / slices);
  c.slices = static_cast<int>((kb0 + c.k_run - 1) / c.k_run);
  c.acc_bytes = (c.pieces > 1 || c.slices > 1) ? align_up(uint64_t(c.slices) * uint64_t(t) * uint64_t(d) * 4, 256) : 0;
  return c;
}

bool rows_map(CUtensorMap* map, const uint16_t* base, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
  return encode_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, cols, rows, ld * 2, 64, box_rows,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

uint64_t linear_ce_workspace(int64_t t, int64_t v, int64_t d, bool backward) {
  if (backward) {
    const CePlan c = ce_plan(t, v, d);
    return c.dz_bytes + c.acc_bytes;
  }
  const uint64_t pieces = 2 * ((uint64_t(v) + kCeTile - 1) / kCeTile);
  return align_up(uint64_t(t) * pieces * 8, 256) + align_up(uint64_t(t) * 4, 256);
}

cudaError_t launch_linear_ce(const CeArgs& a, int num_sms, cudaStream_t s) {
  CUtensorMap th, tw;
  if (!rows_map(&th, a.h, a.d, a.t, a.d, 128) || !rows_map(&tw, a.w, a.d, a.v, a.d, 128)) return cudaErrorInvalidValue;
  CeFwdParams p;
  p.t = static_cast<int>(a.t), p.v = static_cast<int>(a.v), p.d = static_cast<int>(a.d);
  p.pieces = 2 * ((p.v + kCeTile - 1) / kCeTile);
  p.piece = static_cast<float2*>(a.workspace);
  p.hit = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + align_up(uint64_t(a.t) * p.pieces * 8, 256));
  p.targets = a.targets;
  p.status = a.status;
  const cudaError_t e = launch_pair<CfgCeFwd>(th, tw, tw, p, p.t, p.v, num_sms, s, true);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_ce_join, dim3((p.t + 7) / 8), dim3(256), 0, s, p.piece, p.pieces, p.hit, a.targets, p.t, a.v,
                    a.ignore_index, a.loss, a.lse, a.status);
}

cudaError_t launch_linear_ce_bwd(const CeArgs& a, int num_sms, cudaStream_t s) {
  const CePlan c = ce_plan(a.t, a.v, a.d);
  uint16_t* dz = static_cast<uint16_t*>(a.workspace);
  float* acc = c.acc_bytes ? reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + c.dz_bytes) : nullptr;
  int max_clusters = 0;
  cudaError_t e = pair_setup<CfgCeProducts>(num_sms, &max_clusters);
  if (e != cudaSuccess) return e;
  CUtensorMap th, th_mn;
  if (!rows_map(&th, a.h, a.d, a.t, a.d, 128) || !rows_map(&th_mn, a.h, a.d, a.t, a.d, 64))
    return cudaErrorInvalidValue;
  for (int64_t i = 0; i < c.pieces; ++i) {
    const int64_t first = i * c.piece, wide = std::min(c.piece, a.v - first);
    const uint16_t* w = a.w + first * a.d;
    CUtensorMap tw, tw_mn, tz, tz_mn;
    if (!rows_map(&tw, w, a.d, wide, a.d, 128) || !rows_map(&tw_mn, w, a.d, wide, a.d, 64) ||
        !rows_map(&tz, dz, wide, a.t, c.piece, 128) || !rows_map(&tz_mn, dz, wide, a.t, c.piece, 64))
      return cudaErrorInvalidValue;
    CeDzParams z;
    z.t = static_cast<int>(a.t), z.v = static_cast<int>(wide), z.d = static_cast<int>(a.d);
    z.first = first, z.ld = c.piece, z.dz = dz;
    z.targets = a.targets, z.v_all = a.v, z.ignore = a.ignore_index;
    z.lse = a.lse, z.dloss = a.dloss, z.dloss_stride = a.dloss_stride;
    z.status = a.status;
    if ((e = launch_pair<CfgCeDz>(th, tw, tw, z, z.t, z.v, num_sms, s, true)) != cudaSuccess) return e;
    CeProductParams p;
    p.t = z.t, p.v = z.v, p.d = z.d;
    p.k_run = c.k_run;
    p.slices = static_cast<int>(((wide + 63) / 64 + c.k_run - 1) / c.k_run);
    p.mb0 = (p.t + 255) / 256, p.mb1 = (p.v + 255) / 256, p.nb = (p.d + 255) / 256;
    p.dh_first = std::min<int64_t>(c.k_run, (wide + 63) / 64) >= (p.t + 63) / 64;
    p.acc = acc;
    p.add = i > 0;
    p.last = c.slices == 1 && i == c.pieces - 1;
    p.dh = a.dh, p.dw = a.dw + first * a.d;
    p.status = a.status;
    const int64_t tiles = int64_t(CfgCeProducts::tiles0(p)) + CfgCeProducts::tiles1(p);
    const int pairs = static_cast<int>(std::min<int64_t>(tiles, max_clusters));
    e = launch_pdl(k_gemm_pair<CfgCeProducts>, dim3(2 * pairs), dim3(pair_threads<CfgCeProducts>()),
                   pair_smem_bytes<CfgCeProducts>(), s, tz, tw_mn, tz_mn, th_mn, p);
    if (e != cudaSuccess) return e;
  }
  if (c.slices > 1) {
    const int64_t n4 = a.t * a.d / 4;
    return launch_pdl(k_ce_dh, dim3(static_cast<unsigned>((n4 + 255) / 256)), dim3(256), 0, s,
                      reinterpret_cast<const float4*>(acc), c.slices, n4, reinterpret_cast<uint2*>(a.dh));
  }
  return cudaSuccess;
}

}  // namespace sbl
