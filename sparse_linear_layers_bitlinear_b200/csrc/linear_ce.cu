// Softmax cross entropy of a linear head without its logits in memory, on the
// CTA-pair tensor-core GEMM (gemm_pair.cuh).
//
//   z = h w^T,  lse_i = log sum_j exp z_ij,  loss_i = lse_i - z_i,target_i
//   dz_ij = dloss_i (exp(z_ij - lse_i) - [j = target_i]),  dh = dz w,  dw = dz^T h
//
// Forward: a tile of 256 tokens x 256 vocabulary entries leaves, per token, its
// largest logit and the sum of the exponentials below it; a second launch joins
// a token's pieces.  The product bounds it: 2 t v d flops; the exponentials (one
// per logit) run on the epilogue warps under the next tile's product.  Measured,
// sustained (the power cap holds the clock), 8192 x 32768 x 2560: 1020 us, 1350
// TFLOP/s; the library's product alone, with its logits written: 1010 us.
//
// Backward, a piece of the vocabulary at a time, so that dz (the sum of two bf16
// numbers, see below) stays in L2 between its writer and its two readers: a launch
// computes a piece's logits again and writes dz, and runs both products over
// the piece before.  dw rows belong to one piece; dh adds up over the pieces
// in fp32.  With few tokens dh has few output tiles and a long sum over the
// vocabulary, with few entries dw a long one over the tokens; they are then split
// over slices that a last launch joins.
// Measured, sustained, 4096 x 32768 x 2560: 2.85 ms, 1205 TFLOP/s over the five units
// of 687 Gflop that dz's two numbers make of the three, 1.10 of five such products of
// the library (0.52 ms each in the same run).  dh's fp32 sums cost 75 us of it and the
// exponentials 13 (left out of a copy); the rest that is over are dz's way through L2
// and the ends of the launches.
#include <algorithm>
#include <array>
#include <functional>
#include <map>
#include <queue>
#include <utility>
#include <vector>

#include "gemm_launch.cuh"

namespace sbl {

namespace {

constexpr int kCeTile = 256;

// exp(x), relative error about (2 + |x|) 2^-23, results below 2^-126 zero.
__device__ __forceinline__ float exp_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
struct CeFwdParams {
  int t, v, d;
  int pieces;     // per token: one for each vocabulary tile
  float2* piece;  // [t][pieces]: largest logit, sum of exp(logit - largest)
  float* hit;     // [t]: the target's logit
  const int64_t* targets;
  uint32_t* status;
};

// A = h rows, B = w rows, both K-major.  Four epilogue warps, a row a lane: with
// eight, half a tile's columns each, the partial sums double (8192 x 32768 x
// 2560, sustained: 1055 against 1017 us; 63 x 4099 x 512: 9.9 against 10.0).
struct CfgCeFwd {
  using Params = CeFwdParams;
  using Tiles = StripedTiles<CfgCeFwd>;
  static constexpr bool QUANT_X = false, EARLY_TRIGGER = true;
  static constexpr int MAPS = 2;
  static constexpr int EPI_WARPS = 4;
  static constexpr int BN = kCeTile, BK = 64, STAGES = 6;
  static constexpr int A_BYTES = 128 * BK * 2;       // 16 KB
  static constexpr int B_BYTES = (BN / 2) * BK * 2;  // 16 KB
  static constexpr int E_BYTES = 0;
  static constexpr int ACC_COLS = BN;
  static constexpr int TMEM_COLS = 512;
  static constexpr int E_COL0 = 0, E_COLS = 0;
  static constexpr uint32_t IDESC = idesc_bf16(256, BN, false, false);

  __device__ static int rows_M(const Params& p) { return p.t; }
  __device__ static int cols_N(const Params& p) { return p.v; }
  __device__ static int k_blocks(const Params& p) { return (p.d + BK - 1) / BK; }

  // Boxes of 64 rows: with few tokens a box that lies outside h costs less than
  // a part of one (one token, 32768 x 2560: 56 against 71 us with 128 rows).
  __device__ static void load_stage(const CUtensorMap* tA, const CUtensorMap* tB, const CUtensorMap*,
                                    const CUtensorMap*, const Params&, int, uint8_t* sA, uint8_t* sB, uint8_t*, int m0,
                                    int n0, int kb, uint64_t* bar) {
    tma_load_2d_pair(sA, tA, kb * BK, m0, bar);  // [64 rows][64 k] x 2
    tma_load_2d_pair(sA + 8192, tA, kb * BK, m0 + 64, bar);
    tma_load_2d_pair(sB, tB, kb * BK, n0, bar);
    tma_load_2d_pair(sB + 8192, tB, kb * BK, n0 + 64, bar);
  }

  __device__ static void mma_stage(const Params&, int, uint32_t d_tmem, uint32_t, uint8_t* sA, uint8_t* sB, uint8_t*,
                                   bool first) {
    const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB);
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk)
      mma_bf16_pair(d_tmem, smem_desc(a0 + kk * 32, 16, 1024, 2), smem_desc(b0 + kk * 32, 16, 1024, 2), IDESC,
                    (first && kk == 0) ? 0u : 1u);
  }

  __device__ static void epilogue(const Params& p, int, uint32_t t_acc, int row, int n0, int, int, int) {
    const bool in = row < p.t;
    const int64_t target = in ? __ldcg(p.targets + row) : -1;
    float top = -INFINITY, sum = 0.0f;
#pragma unroll 1
    for (int c = 0; c < BN / 32; ++c) {
      const int col0 = n0 + c * 32;
      if (col0 >= p.v) break;  // uniform across the warp
      uint32_t r[32];
      __syncwarp();
      tmem_load_32x32b_x32(t_acc + c * 32, r);
      tmem_load_wait();
      const int left = p.v - col0;
      const int64_t at = target - col0;
      const bool mine = in && at >= 0 && at < 32 && target < p.v;  // the target's logit is in this chunk
      // four maxima and four sums side by side: a single tile's latency is that of these chains
      float z[32], best4[4] = {top, top, top, top}, sum4[4] = {0.0f, 0.0f, 0.0f, 0.0f}, hit = 0.0f;
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        z[e] = e < left ? __uint_as_float(r[e]) : -INFINITY;
        best4[e & 3] = fmaxf(best4[e & 3], z[e]);
        if (mine && e == int(at)) hit += z[e];
      }
      if (mine) p.hit[row] = hit;
      const float best = fmaxf(fmaxf(best4[0], best4[1]), fmaxf(best4[2], best4[3]));
      const float base = best == -INFINITY ? 0.0f : best;
      sum *= exp_of(top - base);
#pragma unroll
      for (int e = 0; e < 32; ++e) sum4[e & 3] += exp_of(z[e] - base);
      sum += (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
      top = best;
    }
    if (in) p.piece[int64_t(row) * p.pieces + n0 / BN] = make_float2(top, sum);
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
// Backward.  One launch works on three kinds of tiles at once, none of which
// needs another's result of the same launch:
//   dz   of the next piece (into the other of two buffers):
//        A = h [t][d], B = the piece's rows of w, both K-major, K = d
//   dh   of this piece:  A = dz [t][v] K-major, B = w's rows MN-major, K = v,
//        in `slices` runs of k_run blocks of 64
//   dw   of this piece:  A = dz MN-major (M = v), B = h MN-major, K = t,
//        in `dw_slices` runs of dw_run blocks
// so that a piece costs one launch and the short tiles fill the gaps that the
// deep ones leave.  Every operand is read in boxes of 64 x 64, which both
// majors can use, so one tensor map each serves h, w and dz (boxes of 128 rows
// for the K-major operands took the same time).
//
// dz, dloss included, is held as the sum of two bf16 numbers: a rounded value and
// what it left, so that it is exact to 2^-16, and both products run over both.  One
// number would cost a rounding as large as the outputs' own wherever an output is
// not ruled by an entry that bf16 holds exactly: over the error of the outputs'
// rounding alone, dh then had 1.01 (flat rows) to 1.44 (median target probability
// 0.63) and dw, whose operand h took dloss with a second rounding, 1.43 to 1.74.
// With two numbers it is 1.00 for both.  The price is five units of product
// instead of three.
constexpr int kCeMaxPairs = 96;
constexpr int kCeMaxTiles = 4096;
constexpr int kCeTileCost = 4;  // of a tile beside its blocks, in blocks: filling the pipe, the last epilogue

struct CeBwdParams {
  CUtensorMap dz_out, dw_out, dh_out;  // of the stores: bf16 boxes of 64 x 32 rows
  CUtensorMap acc_out, dw_sum_out;     // fp32, 32 x 32
  int t, d;
  int zv, vv;           // entries of the next piece (dz) and of this one (dh, dw); 0: none
  int64_t zfirst, vfirst;
  const int64_t* targets;
  int64_t v_all, ignore;
  const float* lse;
  const float* dloss;
  int64_t dloss_stride;
  int lo;               // columns from a dz's rounded value to what it left
  int slices, k_run;        // dh's sum over the vocabulary: blocks of 64 a slice
  int dw_slices, dw_run;    // dw's over the tokens; more than one: fp32 sums of [slices][v up to a multiple of 32][d]
  const float* acc;     // [slices][t up to a multiple of 32][d] fp32 sums of dh, or nullptr: dh is written directly
  int add;              // acc holds the earlier pieces' sum
  int last;             // with one slice: write dh instead of acc
  const uint16_t* h;
  uint16_t* live_h;     // the first launch: where dw's operand goes (else nullptr)
  uint32_t* status;
  int tabled;           // tiles from the table, else striped
  uint16_t sched_off[kCeMaxPairs + 1];
  uint16_t sched[kCeMaxTiles];
};

// EPI epilogue warps: 4, or 8 with half of a tile's columns each where no pair of
// SMs has more than one tile and the epilogue's own time counts (63 x 4099 x 512:
// 18.9 against 20.3 us in a graph; 4 keep a stage more of operands).
template <int EPI>
struct CfgCeBwd {
  using Params = CeBwdParams;
  static constexpr bool QUANT_X = false, EARLY_TRIGGER = true;
  static constexpr int MAPS = 4;
  static constexpr int EPI_WARPS = EPI;
  static constexpr int BN = kCeTile, BK = 64, STAGES = EPI > 4 ? 5 : 6;  // the boxes take the sixth's place
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int B_BYTES = (BN / 2) * BK * 2;
  static constexpr int E_BYTES = 0;
  static constexpr int OUT_BYTES = EPI_WARPS * 2 * 4096;  // two boxes of 32 rows x 128 bytes a warp
  static constexpr int ACC_COLS = BN;
  static constexpr int TMEM_COLS = 512;
  enum { kDz = 0, kDw = 1, kDh = 2 };  // a tile's problem: kind + 4 * slice

  __host__ __device__ static int up(int a, int b) { return (a + b - 1) / b; }
  __host__ __device__ static int tiles_dz(const Params& p) { return up(p.t, 256) * up(p.zv, 256); }
  __host__ __device__ static int tiles_dh(const Params& p) { return p.vv ? up(p.t, 256) * up(p.d, 256) * p.slices : 0; }
  __host__ __device__ static int tiles_dw(const Params& p) { return up(p.vv, 256) * up(p.d, 256) * p.dw_slices; }
  // a product's blocks of 64: those of the rounded dz, then those of what it left
  __host__ __device__ static int depth_dh(const Params& p) { return 2 * up(p.vv, BK); }
  __host__ __device__ static int depth_dw(const Params& p) { return 2 * up(p.t, BK); }

  struct Tiles {
    __device__ static int count(const Params& p, int pair, int npairs) {
      if (p.tabled) return p.sched_off[pair + 1] - p.sched_off[pair];
      const int n = tiles_dz(p) + tiles_dh(p) + tiles_dw(p);
      return pair < n ? (n - pair + npairs - 1) / npairs : 0;
    }
    // Tile numbers: dh, then dw, then dz; the blocks of the same operand rows next to each other.
    __device__ static PairTile at(const Params& p, int pair, int npairs, int i) {
      int id = p.tabled ? p.sched[p.sched_off[pair] + i] : pair + i * npairs;
      const int mt = up(p.t, 256), nd = up(p.d, 256), mv = up(p.vv, 256);
      if (id < tiles_dh(p)) {
        const int slice = id / (mt * nd);
        id -= slice * mt * nd;
        return PairTile{kDh + 4 * slice, id % mt, id / mt, min(depth_dh(p) - slice * p.k_run, p.k_run)};
      }
      id -= tiles_dh(p);
      if (id < tiles_dw(p)) {
        const int slice = id / (mv * nd);
        id -= slice * mv * nd;
        return PairTile{kDw + 4 * slice, id % mv, id / mv, min(depth_dw(p) - slice * p.dw_run, p.dw_run)};
      }
      id -= tiles_dw(p);
      return PairTile{kDz, id % mt, id / mt, up(p.d, BK)};
    }
  };

  // Maps: h, w, this piece's dz, dw's operand of h.
  __device__ static void load_stage(const CUtensorMap* th, const CUtensorMap* tw, const CUtensorMap* tz,
                                    const CUtensorMap* ths, const Params& p, int prob, uint8_t* sA, uint8_t* sB,
                                    uint8_t*, int m0, int n0, int kb, uint64_t* bar) {
    if (prob == kDz) {
      const int k0 = kb * BK, w0 = int(p.zfirst) + n0;
      tma_load_2d_pair(sA, th, k0, m0, bar);  // [64 m][64 k] x 2
      tma_load_2d_pair(sA + 8192, th, k0, m0 + 64, bar);
      tma_load_2d_pair(sB, tw, k0, w0, bar);
      tma_load_2d_pair(sB + 8192, tw, k0, w0 + 64, bar);
    } else if ((prob & 3) == kDw) {
      kb += (prob >> 2) * p.dw_run;
      const int half = up(p.t, BK), k0 = (kb < half ? kb : kb - half) * BK, x = m0 + (kb < half ? 0 : p.lo);
      tma_load_2d_pair(sA, tz, x, k0, bar);  // [64 k][64 m] x 2
      tma_load_2d_pair(sA + 8192, tz, x + 64, k0, bar);
      tma_load_2d_pair(sB, ths, n0, k0, bar);
      tma_load_2d_pair(sB + 8192, ths, n0 + 64, k0, bar);
    } else {
      kb += (prob >> 2) * p.k_run;
      const int half = up(p.vv, BK), k0 = (kb < half ? kb : kb - half) * BK, x = k0 + (kb < half ? 0 : p.lo);
      const int w0 = int(p.vfirst) + k0;
      tma_load_2d_pair(sA, tz, x, m0, bar);  // [64 m][64 k] x 2
      tma_load_2d_pair(sA + 8192, tz, x, m0 + 64, bar);
      tma_load_2d_pair(sB, tw, n0, w0, bar);  // [64 k][64 n] x 2
      tma_load_2d_pair(sB + 8192, tw, n0 + 64, w0, bar);
    }
  }

  // One thread issues every MMA of a pair, so a stage's issue has to stay far
  // below the 512 cycles its MMAs take: the loop over a tile's stages is
  // compiled once for each kind, with constant descriptors.
  static constexpr int MMA_KINDS = 3;
  __device__ static int mma_kind(int prob) { return prob & 3; }
  template <int KIND>
  __device__ static void mma_stage(uint32_t d_tmem, uint8_t* sA, uint8_t* sB, bool first) {
    constexpr bool a_mn = KIND == kDw, b_mn = KIND != kDz;
    const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB);
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk) {
      const uint64_t ad = a_mn ? smem_desc(a0 + kk * 2048, 8192, 1024, 2) : smem_desc(a0 + kk * 32, 16, 1024, 2);
      const uint64_t bd = b_mn ? smem_desc(b0 + kk * 2048, 8192, 1024, 2) : smem_desc(b0 + kk * 32, 16, 1024, 2);
      mma_bf16_pair(d_tmem, ad, bd, idesc_bf16(256, BN, a_mn, b_mn), (first && kk == 0) ? 0u : 1u);
    }
  }

  __device__ static __forceinline__ bool good(const Params& p, int64_t target) {
    return target >= 0 && target < p.v_all && target != p.ignore;
  }

  // The first launch: dw's operand, h with zeros in the rows without loss, whose h
  // may hold anything: zero times a NaN would reach dw.  A row a warp, while the
  // first tiles' products run (4096 x 2560: nothing beside 32768 entries, 2 us
  // beside 1000; loads of several rows at once took no less).
  __device__ static void prologue(const Params& p, int warp, int warps, int lane) {
    if (p.live_h == nullptr) return;
    pdl_wait();  // h and targets may come from the kernel before
    const int vecs = p.d / 8;
    for (int row = warp; row < p.t; row += warps) {
      const bool live = good(p, __ldcg(p.targets + row));
      const uint4* src = reinterpret_cast<const uint4*>(p.h) + int64_t(row) * vecs;
      uint4* dst = reinterpret_cast<uint4*>(p.live_h) + int64_t(row) * vecs;
#pragma unroll 4
      for (int i = lane; i < vecs; i += 32) dst[i] = live ? __ldcg(src + i) : make_uint4(0u, 0u, 0u, 0u);
    }
  }

  // A lane's row of a box (32 words, 128 bytes) goes to shared memory in the
  // 128-byte swizzle, the warp's 32 rows to global memory by one TMA store:
  // whole lines instead of 16 bytes a row (which cost the dz launch a seventh
  // of its time).  Two boxes in turn, from the first one at every tile; the box
  // before the last has been read when this one is filled.
  __device__ static __forceinline__ void put(const CUtensorMap* map, const uint32_t (&word)[32], uint8_t* box, int lane,
                                             int x, int y, bool add) {
    if (lane == 0) bulk_store_wait_read<1>();
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<uint4*>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) =
          make_uint4(word[4 * c], word[4 * c + 1], word[4 * c + 2], word[4 * c + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (add)
        tma_add_2d(map, box, x, y);
      else
        tma_store_2d(map, box, x, y);
      bulk_store_commit();
    }
  }

  // row0: the warp's first row, one row a lane; of the tile's boxes side by side
  // every `parts`-th from `part` on.
  __device__ static void epilogue(const Params& p, int prob, uint32_t t_acc, int row0, int n0, int lane, uint8_t* box,
                                  int part, int parts) {
    int turn = 0;
    const bool dz = prob == kDz, dw = (prob & 3) == kDw;
    const int rows = dw ? p.vv : p.t;
    if (row0 >= rows) return;
    if (lane == 0) bulk_store_wait_read<0>();  // the tile before
    const int row = row0 + lane;
    const bool in = row < rows;
    // fp32 sums.  dh's: stored by the first piece, then added to
    if (dw ? p.dw_slices > 1 : !dz && p.acc != nullptr && !p.last) {
      const int y = (prob >> 2) * up(rows, 32) * 32 + row0;
#pragma unroll 1
      for (int c = part; c < BN / 32; c += parts, turn ^= 4096) {
        uint32_t r[32];
        __syncwarp();
        tmem_load_32x32b_x32(t_acc + c * 32, r);
        tmem_load_wait();
        if (n0 + c * 32 >= p.d) break;
        put(dw ? &p.dw_sum_out : &p.acc_out, r, box + turn, lane, n0 + c * 32, y, !dw && p.add);
      }
      return;
    }
    const int64_t target = !dw && in ? __ldcg(p.targets + row) : p.ignore;
    const bool live = good(p, target);
    if (dz) {
      if (in && !live && target != p.ignore && n0 == 0 && p.zfirst == 0 && part == 0)
        raise_status(p.status, SBL_STATUS_BAD_TARGET);
      dz_tile(p, t_acc, row0, n0, lane, box, part, parts, target, live);
      return;
    }
#pragma unroll 1
    for (int c = part; c < BN / 64; c += parts, turn ^= 4096) {
      const int col0 = n0 + c * 64;
      if (col0 >= p.d) break;  // uniform across the warp
      uint32_t word[32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[32];
        __syncwarp();
        tmem_load_32x32b_x32(t_acc + c * 64 + h * 32, r);
        tmem_load_wait();
        if (!dw && p.add && in) {  // dh's last piece.  Through L2: another SM wrote it in the launch before
          const float* acc = p.acc + int64_t(row) * p.d + col0 + h * 32;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            if (col0 + h * 32 + 4 * q >= p.d) break;
            const float4 a = __ldcg(reinterpret_cast<const float4*>(acc) + q);
            r[4 * q] = __float_as_uint(__uint_as_float(r[4 * q]) + a.x);
            r[4 * q + 1] = __float_as_uint(__uint_as_float(r[4 * q + 1]) + a.y);
            r[4 * q + 2] = __float_as_uint(__uint_as_float(r[4 * q + 2]) + a.z);
            r[4 * q + 3] = __float_as_uint(__uint_as_float(r[4 * q + 3]) + a.w);
          }
        }
        const bool none = !dw && !live;  // a row without loss: zero whatever its sums are (NaN weights)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t u = pack_bf16(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
          word[16 * h + e] = none ? 0u : u;
        }
      }
      put(dw ? &p.dw_out : &p.dh_out, word, box + turn, lane, col0, row0, false);
    }
  }

  __device__ static __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h2 = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h2);
  }

  // dz's tile: of the two boxes one holds the rounded values, the other what they left.
  __device__ static __forceinline__ void dz_tile(const Params& p, uint32_t t_acc, int row0, int n0, int lane,
                                                 uint8_t* box, int part, int parts, int64_t target, bool live) {
    const int row = row0 + lane;
    const float lse = live ? __ldcg(p.lse + row) : 0.0f;
    const float factor = live ? __ldcg(p.dloss + row * p.dloss_stride) : 0.0f;
#pragma unroll 1
    for (int c = part; c < BN / 64; c += parts) {
      const int col0 = n0 + c * 64;
      if (col0 >= p.zv) break;  // uniform across the warp
      if (lane == 0) bulk_store_wait_read<0>();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t r[32];
        __syncwarp();
        tmem_load_32x32b_x32(t_acc + c * 64 + h * 32, r);
        tmem_load_wait();
        const int64_t at = target - p.zfirst - col0 - h * 32;
        const int left = p.zv - col0 - h * 32;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float x = exp_of(__uint_as_float(r[e]) - lse);
          if (at == e) x -= 1.0f;
          const bool none = !live || e >= left;  // columns past the piece are read as part of its last block
          r[e] = none ? 0u : __float_as_uint(x * factor);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t u[4], v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = __uint_as_float(r[8 * q + 2 * e]), y = __uint_as_float(r[8 * q + 2 * e + 1]);
            u[e] = pack_bf16(x, y);
            v[e] = pack_bf16(x - __uint_as_float(u[e] << 16), y - __uint_as_float(u[e] & 0xFFFF0000u));
          }
          uint8_t* dst = box + lane * 128 + (((4 * h + q) ^ (lane & 7)) << 4);
          *reinterpret_cast<uint4*>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
          *reinterpret_cast<uint4*>(dst + 4096) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(&p.dz_out, box, col0, row0);
        tma_store_2d(&p.dz_out, box + 4096, col0 + p.lo, row0);
        bulk_store_commit();
      }
    }
  }
};

// The slices of dh and of dw added in their order, 4 elements a thread.
struct CeSum {
  const float4* part;  // [slices][slice_n4]
  int slices;
  int64_t slice_n4, n4;  // n4 0: not split, nothing to do
  uint2* out;
};

__global__ void __launch_bounds__(256)
    k_ce_sum(const CeSum dh, const CeSum dw, unsigned dh_blocks, int row_n4, const int64_t* __restrict__ targets,
             int64_t v, int64_t ignore) {
  pdl_wait();
  pdl_trigger();
  const bool first = blockIdx.x < dh_blocks;
  const CeSum& s = first ? dh : dw;
  const int64_t i = int64_t(blockIdx.x - (first ? 0u : dh_blocks)) * 256 + threadIdx.x;
  if (i >= s.n4) return;
  bool live = true;
  if (first) {
    const int64_t target = targets[i / row_n4];
    live = target >= 0 && target < v && target != ignore;
  }
  float4 a = __ldcg(s.part + i);
  for (int k = 1; k < s.slices; ++k) {
    const float4 b = __ldcg(s.part + k * s.slice_n4 + i);
    a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(a.z, a.w);
  s.out[i] = live ? make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi))
                  : make_uint2(0u, 0u);
}

// How the backward pass cuts its work.
constexpr int64_t kCeDzBytes = int64_t(64) << 20;  // dz of one piece of several: half of L2
// A piece's least width, which counts above 8192 tokens: dh's sums (4 t d bytes, past
// L2 there) are read and written once a piece, so narrow pieces cost more than a dz
// that leaves L2.  256, 1024, 2048 and 4096 entries: 32768 x 151936 x 3584 198, 180, 170
// and 171 ms; 32768 x 32768 x 2560 30.7, 25.7, 24.1, 24.9; 131072 x 32768 x 1024 184, 69, 51, 47.
constexpr int64_t kCeMinPiece = 2048;

struct CePlan {
  int64_t piece;    // vocabulary entries of a piece, a multiple of 256
  int64_t pieces;
  int slices, k_run, dw_slices, dw_run;
  int64_t acc_rows, dw_rows;  // rows of a slice of the sums: t and v up to a multiple of the 32 that a store writes
  uint64_t dz_bytes, acc_bytes, dw_bytes, live_h_bytes;  // dz: one buffer of two (one piece: of one)
  uint64_t total() const { return dz_bytes * (pieces > 1 ? 2 : 1) + acc_bytes + dw_bytes + live_h_bytes; }
};

CePlan ce_plan(int64_t t, int64_t v, int64_t d) {
  CePlan c;
  const int64_t padded = (v + 255) / 256 * 256;
  // one piece needs one buffer: it may be as large as the two of several
  const int64_t bytes = t * padded * 4 <= 2 * kCeDzBytes ? 2 * kCeDzBytes : kCeDzBytes;
  const int64_t most = std::max(bytes / (4 * t) / 256 * 256, kCeMinPiece);
  c.pieces = (padded + most - 1) / most;
  c.piece = ((padded / 256 + c.pieces - 1) / c.pieces) * 256;  // even pieces
  c.pieces = (padded + c.piece - 1) / c.piece;
  c.dz_bytes = align_up(uint64_t(t) * uint64_t(c.piece) * 4, 256);
  c.live_h_bytes = align_up(uint64_t(t) * uint64_t(d) * 2, 256);
  // A dh tile is as deep as the piece is wide, a dw tile as there are tokens.  A
  // run of the sum is about what each pair of SMs has to do anyway (or 8 blocks).
  // dw is split where it has few tiles (one piece) and would take twice as long
  // (4096 x 256 x 2560: 69 -> 48 us, 16384 x 256 x 1024: 205 -> 71).
  const int64_t nb = (d + 255) / 256, mb0 = (t + 255) / 256, mb1 = c.piece / 256;
  const int64_t kb0 = (std::min(c.piece, v) + 63) / 64 * 2, kb1 = (t + 63) / 64 * 2;
  const int64_t pairs = 74;  // 148 SMs
  const int64_t share = std::max<int64_t>((mb0 * nb * kb0 + mb1 * nb * kb1) / pairs, 8);
  int64_t slices = std::min<int64_t>((kb0 + share - 1) / share, 32);
  c.k_run = static_cast<int>((kb0 + slices - 1) / slices);
  c.slices = static_cast<int>((kb0 + c.k_run - 1) / c.k_run);
  c.acc_rows = (t + 31) / 32 * 32;
  const uint64_t acc = uint64_t(c.slices) * uint64_t(c.acc_rows) * uint64_t(d) * 4;
  const int64_t dw_slices = c.pieces > 1 ? 1 : std::min<int64_t>(std::max<int64_t>(kb1 / share, 1), 32);
  c.dw_run = static_cast<int>((kb1 + dw_slices - 1) / dw_slices);
  c.dw_slices = static_cast<int>((kb1 + c.dw_run - 1) / c.dw_run);
  c.dw_rows = (v + 31) / 32 * 32;
  c.dw_bytes = c.dw_slices > 1 ? align_up(uint64_t(c.dw_slices) * uint64_t(c.dw_rows) * uint64_t(d) * 4, 256) : 0;
  c.acc_bytes = c.pieces > 1 || c.slices > 1 ? align_up(acc, 256) : 0;
  return c;
}

// The tiles of one launch over the pairs, deepest first, each to the pair with
// the least work so far, written into p.  Cached per shape.
struct CeSchedule {
  std::vector<uint16_t> off, ids;
};

void ce_schedule(int n_dh, int k_dh, int n_dw, int k_dw, int n_dz, int k_dz, int npairs, CeBwdParams& p) {
  static std::mutex mu;
  static std::map<std::array<int, 7>, CeSchedule> cache;
  std::lock_guard<std::mutex> lock(mu);
  const std::array<int, 7> key = {n_dh, k_dh, n_dw, k_dw, n_dz, k_dz, npairs};
  const auto use = [&p](const CeSchedule& sch) {
    std::copy(sch.off.begin(), sch.off.end(), p.sched_off);
    std::copy(sch.ids.begin(), sch.ids.end(), p.sched);
  };
  const auto it = cache.find(key);
  if (it != cache.end()) return use(it->second);
  struct Kind {
    int first, n, depth;
  };
  Kind kinds[3] = {{0, n_dh, k_dh}, {n_dh, n_dw, k_dw}, {n_dh + n_dw, n_dz, k_dz}};
  std::stable_sort(kinds, kinds + 3, [](const Kind& a, const Kind& b) { return a.depth > b.depth; });
  std::vector<std::vector<uint16_t>> per(npairs);
  using Load = std::pair<int64_t, int>;  // work so far, pair
  std::priority_queue<Load, std::vector<Load>, std::greater<Load>> least;
  for (int q = 0; q < npairs; ++q) least.push({0, q});
  for (const Kind& k : kinds)
    for (int i = 0; i < k.n; ++i) {
      const Load l = least.top();
      least.pop();
      per[l.second].push_back(static_cast<uint16_t>(k.first + i));
      least.push({l.first + k.depth + kCeTileCost, l.second});
    }
  CeSchedule sch;
  sch.off.push_back(0);
  for (const auto& ids : per) {
    sch.ids.insert(sch.ids.end(), ids.begin(), ids.end());
    sch.off.push_back(static_cast<uint16_t>(sch.ids.size()));
  }
  use(sch);
  if (cache.size() >= 512) cache.clear();  // 8 KB each at most
  cache.emplace(key, std::move(sch));
}

bool rows_map(CUtensorMap* map, const uint16_t* base, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
  return encode_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, cols, rows, ld * 2, 64, box_rows,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

uint64_t linear_ce_workspace(int64_t t, int64_t v, int64_t d, bool backward) {
  if (backward) return ce_plan(t, v, d).total();
  const uint64_t pieces = (uint64_t(v) + kCeTile - 1) / kCeTile;
  return align_up(uint64_t(t) * pieces * 8, 256) + align_up(uint64_t(t) * 4, 256);
}

namespace {

template <int EPI>
cudaError_t launch_ce_tiles(const CUtensorMap& th, const CUtensorMap& tw, const CUtensorMap& tz, const CUtensorMap& ths,
                            const CeBwdParams& p, int pairs, int num_sms, cudaStream_t s) {
  using Cfg = CfgCeBwd<EPI>;
  int max_clusters = 0;
  const cudaError_t e = pair_setup<Cfg>(num_sms, &max_clusters);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_gemm_pair<Cfg>, dim3(2 * pairs), dim3(pair_threads<Cfg>()), pair_smem_bytes<Cfg>(), s, th, tw, tz,
                    ths, p);
}

}  // namespace

cudaError_t launch_linear_ce(const sbl_linear_ce_args& a, int num_sms, cudaStream_t s) {
  const uint16_t *h = static_cast<const uint16_t*>(a.h), *w = static_cast<const uint16_t*>(a.w);
  CUtensorMap th, tw;
  if (!rows_map(&th, h, a.d, a.t, a.d, 64) || !rows_map(&tw, w, a.d, a.v, a.d, 64)) return cudaErrorInvalidValue;
  CeFwdParams p;
  p.t = static_cast<int>(a.t), p.v = static_cast<int>(a.v), p.d = static_cast<int>(a.d);
  p.pieces = (p.v + kCeTile - 1) / kCeTile;
  p.piece = static_cast<float2*>(a.workspace);
  p.hit = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + align_up(uint64_t(a.t) * p.pieces * 8, 256));
  p.targets = a.targets;
  p.status = a.status_dev;
  const cudaError_t e = launch_pair<CfgCeFwd>(th, tw, tw, p, p.t, p.v, num_sms, s, true);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_ce_join, dim3((p.t + 7) / 8), dim3(256), 0, s, p.piece, p.pieces, p.hit, a.targets, p.t, a.v,
                    a.ignore_index, a.loss, a.lse, a.status_dev);
}

cudaError_t launch_linear_ce_bwd(const sbl_linear_ce_backward_args& a, int num_sms, cudaStream_t s) {
  const CePlan c = ce_plan(a.t, a.v, a.d);
  const uint16_t *h = static_cast<const uint16_t*>(a.h), *w = static_cast<const uint16_t*>(a.w);
  uint16_t *dh = static_cast<uint16_t*>(a.dh), *dw = static_cast<uint16_t*>(a.dw);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  uint16_t* dz[2] = {reinterpret_cast<uint16_t*>(ws),
                     reinterpret_cast<uint16_t*>(ws + (c.pieces > 1 ? c.dz_bytes : 0))};
  ws += c.dz_bytes * (c.pieces > 1 ? 2 : 1);
  float* acc = c.acc_bytes ? reinterpret_cast<float*>(ws) : nullptr;
  ws += c.acc_bytes;
  float* dw_sum = c.dw_bytes ? reinterpret_cast<float*>(ws) : nullptr;
  ws += c.dw_bytes;
  uint16_t* live_h = reinterpret_cast<uint16_t*>(ws);  // dw's operand
  cudaError_t e;
  int max_clusters = 0;
  if ((e = pair_setup<CfgCeBwd<4>>(num_sms, &max_clusters)) != cudaSuccess) return e;
  CUtensorMap th, tw, ths, dh_out, acc_out, dw_sum_out;
  if (acc != nullptr && !encode_tmap_2d(&acc_out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, acc, a.d, c.slices * c.acc_rows,
                                        a.d * 4, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if (dw_sum != nullptr && !encode_tmap_2d(&dw_sum_out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dw_sum, a.d,
                                           c.dw_slices * c.dw_rows, a.d * 4, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if (!rows_map(&dh_out, dh, a.d, a.t, a.d, 32) || !rows_map(&th, h, a.d, a.t, a.d, 64) ||
      !rows_map(&tw, w, a.d, a.v, a.d, 64) || !rows_map(&ths, live_h, a.d, a.t, a.d, 64))
    return cudaErrorInvalidValue;
  const auto wide = [&](int64_t i) { return i < 0 || i >= c.pieces ? 0 : std::min(c.piece, a.v - i * c.piece); };
  for (int64_t i = -1; i < c.pieces; ++i) {  // dz of piece i + 1, products of piece i
    using Cfg = CfgCeBwd<4>;
    CeBwdParams p;
    p.t = static_cast<int>(a.t), p.d = static_cast<int>(a.d);
    p.zv = static_cast<int>(wide(i + 1)), p.zfirst = (i + 1) * c.piece;
    p.vv = static_cast<int>(wide(i)), p.vfirst = i * c.piece;
    p.targets = a.targets, p.v_all = a.v, p.ignore = a.ignore_index;
    p.lse = a.lse, p.dloss = a.dloss, p.dloss_stride = a.dloss_stride;
    p.lo = static_cast<int>(c.piece);
    p.k_run = c.k_run, p.dw_slices = c.dw_slices, p.dw_run = c.dw_run;
    p.slices = (Cfg::depth_dh(p) + c.k_run - 1) / c.k_run;
    p.acc = acc;
    p.add = i > 0;
    p.last = c.slices == 1 && i == c.pieces - 1;
    p.h = h, p.live_h = i < 0 ? live_h : nullptr;
    p.status = a.status_dev;
    CUtensorMap tz = th;
    p.dz_out = p.dw_out = p.acc_out = p.dw_sum_out = p.dh_out = dh_out;
    const auto dz_map = [&](CUtensorMap* map, int64_t j, int box_rows) {
      return rows_map(map, dz[j & 1], 2 * c.piece, a.t, 2 * c.piece, box_rows);
    };
    if (p.zv > 0 && !dz_map(&p.dz_out, i + 1, 32)) return cudaErrorInvalidValue;
    if (p.vv > 0 && (!dz_map(&tz, i, 64) ||
                     !rows_map(&p.dw_out, dw + p.vfirst * a.d, a.d, p.vv, a.d, 32)))
      return cudaErrorInvalidValue;
    if (acc != nullptr) p.acc_out = acc_out;
    if (dw_sum != nullptr) p.dw_sum_out = dw_sum_out;
    const int n_dh = Cfg::tiles_dh(p), n_dw = Cfg::tiles_dw(p), n_dz = Cfg::tiles_dz(p);
    const int64_t tiles = int64_t(n_dh) + n_dw + n_dz;
    // the first launch has a warp for each row to copy too, if need be on pairs without a tile
    const int64_t busy = i < 0 ? std::max<int64_t>(tiles, (a.t + 7) / 8) : tiles;
    const int pairs = static_cast<int>(std::min<int64_t>({busy, max_clusters, kCeMaxPairs}));
    p.tabled = tiles <= kCeMaxTiles;
    if (p.tabled)
      ce_schedule(n_dh, std::min(c.k_run, Cfg::depth_dh(p)), n_dw, std::min(c.dw_run, Cfg::depth_dw(p)), n_dz,
                  (p.d + 63) / 64, pairs, p);
    e = tiles <= pairs ? launch_ce_tiles<8>(th, tw, tz, ths, p, pairs, num_sms, s)
                       : launch_ce_tiles<4>(th, tw, tz, ths, p, pairs, num_sms, s);
    if (e != cudaSuccess) return e;
  }
  if (c.slices > 1 || c.dw_slices > 1) {
    CeSum h_sum{reinterpret_cast<const float4*>(acc), c.slices, c.acc_rows * a.d / 4, 0, reinterpret_cast<uint2*>(dh)};
    CeSum w_sum{reinterpret_cast<const float4*>(dw_sum), c.dw_slices, c.dw_rows * a.d / 4, 0,
                reinterpret_cast<uint2*>(dw)};
    if (c.slices > 1) h_sum.n4 = a.t * a.d / 4;
    if (c.dw_slices > 1) w_sum.n4 = a.v * a.d / 4;
    const unsigned h_blocks = static_cast<unsigned>((h_sum.n4 + 255) / 256),
                   w_blocks = static_cast<unsigned>((w_sum.n4 + 255) / 256);
    return launch_pdl(k_ce_sum, dim3(h_blocks + w_blocks), dim3(256), 0, s, h_sum, w_sum, h_blocks,
                      static_cast<int>(a.d / 4), a.targets, a.v, a.ignore_index);
  }
  return cudaSuccess;
}

}  // namespace sbl
