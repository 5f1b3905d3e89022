// Softmax cross-entropy of hidden states against an LM head, in pieces of the
// vocabulary, without keeping the logits (the loss of a drafter's training, paper
// section 4.2, eq. 1, from the hidden states on):
//
//   z = H W' / T      lse_r = ln sum_v e^(z_rv)      loss_r = lse_r - z_r,target
//   G = d_loss / T (e^(z - lse) - 1[v = target])     dH = G W     dW = G' H
//
// Rows whose target lies outside the vocabulary have no loss; the first kernel
// packs the other rows' hidden states (whatever their alignment and stride), so
// that nothing is computed for the ignored rows and nothing that they hold (NaN
// from uninitialised padding) reaches a sum over rows.  How many are kept is known
// on the device alone: grids are sized for all rows, and CTAs take items while
// there are any.
//
// One GEMM kernel with these uses:
//   stats    z of a tile of rows x vocabulary columns, reduced in registers to a
//            (maximum, sum) pair a row and half tile, and the target's z
//   grad     z again, turned into G: a piece of it is stored, rounded to bf16
//   hidden   dH += G W over a piece (W read with its vocabulary axis along K)
//   weight   dW = G' H of a piece's rows of the head (both along the rows)
//   grads    the last two in one launch, where both are small (choosing between them
//            tile by tile costs large ones 5 %)
// A piece is as many columns as keep G within kPieceBytes.
//
// bf16: the two CTAs of a cluster share a tile of 256 x 256 (tcgen05 cta_group::2, each
// holding half of either operand); a thread of each loads tiles by TMA into a ring, a
// warp of the first issues the MMAs, eight warps of each read the sums.  The tensor
// cores' fp32 sums truncate (by 2e-8 of the sum a step of 16, to one side), which over a
// dim of 4,096 would put the loss off by 3e-6 of itself; so a sum ends after kSumBlocks
// blocks of 64 and the eight warps add it to fp32 registers, two accumulators taking
// turns.
//
// fp32 tensors enter as three bf16 planes each (x = h + m + l, 24 bits), every
// product as six (h h, h m, m h, m m, h l, l h; what is left out is below 2^-24),
// the five small ones with a sum of their own that spans more blocks.  One CTA a tile
// of 128 x 128.  The head's planes exist in shared memory alone: eight more warps read
// its fp32 rows a block ahead into registers and write the planes where the MMAs take
// them.  (28 rows of 2,824 against 129,969: 457 us, with a copy of the planes in memory
// 1,343; the head's 1.47 GB read once are 219.)
//
// Bounds.  Many rows: the tensor cores.  2,048 x 4,096 x 22,016: the loss at 1.89
// PFLOP/s (pipe active in 97 % of the cycles), the gradient's three products at 1.83,
// 1.72 and 1.74; 8,192 x 4,096 x 151,936 back to back 5.5 ms, at the power cap.  Few rows:
// HBM, the head once for the loss (15 x 4,096 x 151,936: 198 us, 6.3 TB/s) and twice for a
// gradient (44 x 4,240 x 94,344, both: 435 us).  A dim of a few hundred: the epilogue
// (6,113 x 136 x 50,082: loss 107 us, of which the MMAs 44).  fp32: shared memory, which
// the six products read planes from (a block of 64 takes 2,600 cycles, 1,536 of them
// MMAs); 333 x 256 x 8,705 gradients in 51 to 60 us.
#include <cuda.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "cross_entropy.cuh"
#include "gemm.cuh"
#include "ptx.cuh"

namespace dflash {
namespace {

constexpr int kBM = 128;                 // rows of a CTA's part of a tile: the lanes of tensor memory
constexpr int kEpiWarps = 8;
constexpr int kConvWarps = 8;            // fp32: warps that turn the head into planes
template <int PL> constexpr int gemm_threads() { return 128 + 32 * kEpiWarps + (PL == 3 ? 32 * kConvWarps : 0); }
constexpr long long kBudget = 400000000LL;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTailWaves = 3;   // waves of parts of cut tiles (the hidden states' gradient), at most
constexpr int kDirectPiece = 1024;
constexpr size_t kPieceBytes = size_t(192) << 20;

enum Use { kStats, kGrad, kHidden, kWeight, kGrads };

// PL planes; G CTAs share a tile of BN columns.
template <int PL, int G, int BN>
struct GemmCfg {
  static constexpr int kCtas = G;
  static constexpr int kTM = kBM * kCtas, kBN = BN;   // the tile
  static constexpr int kOwnN = kBN / kCtas;                // rows of the second operand that a CTA holds
  static constexpr int kA = kBM * 128, kB = kOwnN * 128;   // bytes of a K block of 64
  static constexpr int kStage = PL * (kA + kB);
  static constexpr int kStages = PL == 3 ? 2 : kOwnN == 128 ? 6 : 4;
  static constexpr int kOut = kEpiWarps * 4096;            // rows staged on their way out, 32 x 64 a warp
  static constexpr int kAccCols = kBN;                     // tensor-memory columns of an accumulator
  static constexpr int kNC = kBN / 2;                      // columns of an epilogue thread
  static constexpr int kSumBlocks = PL == 1 ? 8 : 2;       // K blocks that one sum of the tensor cores spans
  static constexpr int kSmallSums = 4;                     // three planes: sums of the large product to one of the small ones
  static constexpr size_t kBytes = 1024 + (size_t)kStages * kStage + kOut + 256;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int PL> struct Tensor { using T = float; };
template <> struct Tensor<1> { using T = __nv_bfloat16; };

struct GemmArgs {
  CePlan pl;
  int v0, cols;          // the piece's first vocabulary column, how many there are
  int first;             // hidden: the sums start here
  float scale2, scale2_lo;   // log2(e) / T and its rounding residual
  const void* weight;
  void* d_hidden;
  int64_t d_row_stride;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// two fp32 values at once
__device__ __forceinline__ uint64_t two(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void split2(uint64_t r, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// ---------------------------------------------------------------- planes
// Two values as a register of two bf16, the first in the lower half.
__device__ __forceinline__ uint32_t pack_rn(float x, float y) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_rz(float x, float y) {
  uint32_t r;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Eight values as planes `stride` elements apart, 16 bytes each: rounded to one bf16, or as
// three whose sum has all 24 bits (the first one cut off, so that no finite value rounds
// to infinity).
template <int PL>
__device__ __forceinline__ void put8(__nv_bfloat16* dst, size_t stride, const float* v) {
  uint32_t w[PL][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float x = v[2 * j], y = v[2 * j + 1];
    if constexpr (PL == 1) {
      w[0][j] = pack_rn(x, y);
    } else {
      w[0][j] = pack_rz(x, y);
      x -= low_of(w[0][j]);
      y -= high_of(w[0][j]);
      w[1][j] = pack_rn(x, y);
      w[2][j] = pack_rn(x - low_of(w[1][j]), y - high_of(w[1][j]));
    }
  }
#pragma unroll
  for (int k = 0; k < PL; ++k) *reinterpret_cast<uint4*>(dst + k * stride) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
}
// Eight values at p; `vec`: whether 16-byte accesses may be used.
__device__ __forceinline__ void get8(const float* p, bool vec, float* v) {
  if (vec) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = p[j];
  }
}
__device__ __forceinline__ void get8(const __nv_bfloat16* p, bool vec, float* v) {
  if (vec) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = __uint_as_float(w[j] << 16), v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __bfloat162float(p[j]);
  }
}
__device__ __forceinline__ void set8(float* p, bool vec, const float* v) {
  if (vec) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = v[j];
  }
}
__device__ __forceinline__ void set8(__nv_bfloat16* p, bool vec, const float* v) {
  if (vec) {
    put8<1>(p, 0, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = __float2bfloat16_rn(v[j]);
  }
}
// Eight values plus f times those at p (16-byte aligned).
template <typename T>
__device__ __forceinline__ void add_rest(const T* p, float f, float* v) {
  float w[8];
  get8(p, true, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = fmaf(f, w[j], v[j]);
}
template <typename T>
__device__ __forceinline__ bool rows_vec(const T* p, int64_t stride) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(stride * (int64_t)sizeof(T))) & 15) == 0;
}

// The parts of a cut tile that cost least, in K blocks: their waves, each with a start and
// an end worth 8, and their sums' way through memory.  A warp tries all.
__device__ __forceinline__ int parts_of_cut(const CePlan& pl, int kept, int groups) {
  const int tiles = (kept + pl.tile - 1) / pl.tile * ((pl.dim + pl.bn - 1) / pl.bn), rest = tiles % groups, all = pl.piece / 64;
  const int p = (threadIdx.x & 31) + 1;
  float cost = 1e30f;
  if (p == 1) cost = all + 8.f;
  else if (!pl.direct && rest && rest * p <= kTailWaves * groups && p * 4 <= all)
    cost = ((rest * p + groups - 1) / groups) * ((float)all / p + 8.f) + 8.f * rest * p / groups;
  const unsigned least = __reduce_min_sync(0xffffffffu, __float_as_uint(cost));   // (costs are positive)
  return __ffs(__ballot_sync(0xffffffffu, __float_as_uint(cost) == least));
}

// ---------------------------------------------------------------- rows that count
// Kept rows in their order: where each came from, its target and statistics, and
// its hidden state as planes.  Every CTA counts the kept rows before its own.
// Ignored rows get their results here: loss and lse 0, or a gradient of zeros.
// Latency for few rows (7 us for 777 x 2,560 alone), then HBM (4,096 x 4,096: 20 us).
constexpr int kGatherThreads = 256;

template <typename T, int PL, bool BWD>
__global__ void __launch_bounds__(kGatherThreads) ce_gather_kernel(CePlan pl, CeTensors t, int per, int groups) {
  griddep_wait();
  griddep_trigger();
  __shared__ int s_before, s_total, s_warp[kGatherThreads / 32], s_list[kGatherThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_before = s_total = 0;
  __syncthreads();
  const int r0 = min((int)blockIdx.x * per, pl.rows), r1 = min(r0 + per, pl.rows);
  auto inside = [&](int r) { return (unsigned)t.targets[r] < (unsigned)pl.vocab; };
  int before = 0, total = 0;
  for (int r = tid; r < pl.rows; r += kGatherThreads) {
    const int in = inside(r);
    total += in;
    before += in && r < r0;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) {
    atomicAdd(&s_before, before);
    atomicAdd(&s_total, total);
  }
  __syncthreads();
  before = s_before;
  total = s_total;
  if (blockIdx.x == 0 && warp == 0) {
    const int parts = BWD ? parts_of_cut(pl, total, groups) : 1;
    if (lane == 0) {
      *pl.status = 0;
      pl.kept[0] = total;
      pl.kept[1] = parts;
    }
  }
  const T* hidden = static_cast<const T*>(t.hidden);
  T* d_hidden = static_cast<T*>(t.d_hidden);
  const bool vec = rows_vec(hidden, t.row_stride), d_vec = BWD && rows_vec(d_hidden, t.d_row_stride);
  const size_t plane = (size_t)pl.rows_pad * pl.dim_pad;
  const float zero[8] = {};
  for (int base = r0; base < r1; base += kGatherThreads) {
    const int r = base + tid, n = min(kGatherThreads, r1 - base);
    const bool in = r < r1 && inside(r);
    const unsigned votes = __ballot_sync(0xffffffffu, in);
    if (lane == 0) s_warp[warp] = __popc(votes);
    __syncthreads();
    int at = before + __popc(votes & ((1u << lane) - 1)), here = 0;
    for (int w = 0; w < kGatherThreads / 32; ++w) {
      if (w < warp) at += s_warp[w];
      here += s_warp[w];
    }
    if (tid < n) s_list[tid] = in ? at : -1;
    if (in) {
      pl.row_of[at] = r;
      pl.target[at] = t.targets[r];
      if (BWD) {
        const double l = (double)t.lse_in[r] * 1.4426950408889634074;
        pl.lse2[at] = make_float2((float)l, (float)(l - (double)(float)l));
        pl.gain[at] = t.d_loss[r] / t.temperature;
      }
    } else if (r < r1 && !BWD) {
      t.loss[r] = 0.f;
      t.lse[r] = 0.f;
    }
    __syncthreads();
    for (int i = warp; i < n; i += kGatherThreads / 32) {
      const int to = s_list[i];
      if (to >= 0) {
        const T* src = hidden + (int64_t)(base + i) * t.row_stride;
        __nv_bfloat16* dst = pl.h + (size_t)to * pl.dim_pad;
        constexpr int U = PL == 1 ? 8 : 4;
        for (int c0 = lane * 8; c0 < pl.dim_pad; c0 += 256 * U) {
          float v[U][8] = {};
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (c0 + u * 256 < pl.dim) get8(src + c0 + u * 256, vec, v[u]);
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (c0 + u * 256 < pl.dim_pad) put8<PL>(dst + c0 + u * 256, plane, v[u]);
        }
      } else if (BWD && d_hidden) {
        T* dst = d_hidden + (int64_t)(base + i) * t.d_row_stride;
        for (int c = lane * 8; c < pl.dim; c += 256) set8(dst + c, d_vec, zero);
      }
    }
    before += here;
    __syncthreads();
  }
  // the last tile's rows behind the kept ones
  const int end = min((total + pl.tile - 1) / pl.tile * pl.tile, pl.rows_pad);
  for (int p = total + blockIdx.x * (kGatherThreads / 32) + warp; p < end; p += gridDim.x * (kGatherThreads / 32)) {
    __nv_bfloat16* dst = pl.h + (size_t)p * pl.dim_pad;
    for (int c = lane * 8; c < pl.dim_pad; c += 256) put8<PL>(dst + c, plane, zero);
  }
}

// ---------------------------------------------------------------- tensor-core pieces
// High word of every shared-memory descriptor: 128-byte swizzle, 8 rows are 1024 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// K-major: a row's 64 values run along K.  MN-major: they run along M or N, the
// rows along K, and the tile of the next 64 is 64 rows further.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, bool mn) {
  return (addr >> 4) | ((mn ? 8192u >> 4 : 1u) << 16);
}
__host__ __device__ constexpr uint32_t k_step(bool mn) { return mn ? 16 * 128 >> 4 : 32 >> 4; }   // 16 along K

__device__ __forceinline__ bool elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
// ---- forms for a CTA alone (G = 1) and for a pair (G = 2)
template <int G>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (G == 2) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
// One arrival at `bar` (of both CTAs of a pair) when what this thread issued completes.
template <int G>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (G == 2)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     ptx::smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
  else
    ptx::mma_commit(bar);
}
// The same for this CTA's barrier alone.
template <int G>
__device__ __forceinline__ void commit_own(uint64_t* bar) {
  if constexpr (G == 2)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
  else
    ptx::mma_commit(bar);
}
template <int G>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot) {
  if constexpr (G == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(ptx::smem_u32(slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    ptx::tmem_alloc(slot, 512);
    ptx::tmem_relinquish();
  }
}
template <int G>
__device__ __forceinline__ void tmem_free(uint32_t taddr) {
  if constexpr (G == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
  else ptx::tmem_dealloc(taddr, 512);
}
// The same place in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(ptx::smem_u32(p)), "r"(rank));
  return r;
}
// Box (x = column, y = row) of a tensor map into this CTA's shared memory; the bytes
// count at `bar`, an address in the cluster (the pair's first CTA).
template <int G>
__device__ __forceinline__ void tma_tile(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  if constexpr (G == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
  else
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                     ptx::smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\tcp.async.bulk.commit_group;" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(ptx::smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}
// Arrival at a barrier of the pair's first CTA.  It says that this warp has read its part of
// tensor memory (tcgen05.wait::ld and the fence before it see to that) and hands over no
// other memory, so it releases at the scope of the CTA: at the cluster's it would wait for
// the epilogue's global stores at every sum.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// As ptx::mbar_try_wait, for what a thread of the other CTA did before it arrived.
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(ptx::smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// 32 columns of this warp's lanes; used after tmem_loaded.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
// Waits for this thread's loads; no use of the n values moves before it.
template <int N>
__device__ __forceinline__ void tmem_loaded(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int j = 0; j < N; ++j) asm volatile("" : "+f"(v[j]));
}
template <int G>
__device__ __forceinline__ void sync_tile_ctas() {
  if constexpr (G == 2) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
}
__device__ __forceinline__ void red_add4(float* p, float a, float b, float c, float d) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

// Items of a launch, for a group of CTAs that shares a tile: output tiles with their K
// blocks of 64.
//
// The hidden states' gradient has few tiles and a long K: the tiles that would not
// fill the last wave of CTAs are cut along K into as many parts as make that wave
// shortest; each part has its sums in memory of its own, and they are added in order
// at the end.  The head's gradient (many short tiles) comes behind.
template <int PL, int G, int BN, int USE>
struct Items {
  using C = GemmCfg<PL, G, BN>;
  int m_tiles, n_tiles, blocks;
  int whole, parts;   // tiles that are not cut; parts of each of the others
  int w_from, w_n, w_blocks, n;   // first item, column tiles and blocks of the head's gradient; all items
  __device__ __forceinline__ Items(const GemmArgs& a, int kept, int groups) {
    const CePlan& pl = a.pl;
    m_tiles = (kept + C::kTM - 1) / C::kTM;
    constexpr bool kGradient = USE == kHidden || USE == kWeight || USE == kGrads;
    n_tiles = ((kGradient ? pl.dim : a.cols) + C::kBN - 1) / C::kBN;
    blocks = kGradient ? (a.cols + 63) / 64 : pl.dim_pad / 64;
    parts = USE == kHidden || USE == kGrads ? pl.kept[1] : 1;
    whole = m_tiles * n_tiles;
    const int rest = parts > 1 ? whole % groups : 0;
    whole -= rest;
    n = whole + rest * parts;
    if (USE == kWeight || USE == kGrads) {
      if (USE == kWeight) n = 0;
      w_from = n;
      w_n = n_tiles;
      w_blocks = (kept + 63) / 64;
      n += (a.cols + C::kTM - 1) / C::kTM * w_n;
    }
  }
  __device__ __forceinline__ bool weight(int item) const { return USE == kWeight || (USE == kGrads && item >= w_from); }
  // first row and column of the item's tile, and its K blocks
  __device__ __forceinline__ void get(int item, int& m0, int& n0, int& b0, int& b1) const {
    b0 = 0;
    if (weight(item)) {   // along a row of tiles: G's columns stay in L2
      const int tile = item - w_from;
      n0 = tile % w_n * C::kBN;
      m0 = tile / w_n * C::kTM;
      b1 = w_blocks;
      return;
    }
    int tile = item;
    b1 = blocks;
    if ((USE == kHidden || USE == kGrads) && item >= whole) {   // the same part of all tiles side by side
      const int rest = m_tiles * n_tiles - whole, part = (item - whole) / rest;
      tile = whole + (item - whole) - part * rest;
      b0 = (int)((long long)blocks * part / parts);
      b1 = (int)((long long)blocks * (part + 1) / parts);
    }
    m0 = tile % m_tiles * C::kTM;
    n0 = tile / m_tiles * C::kBN;
  }
};

struct GemmBars {
  uint64_t full[6], empty[6], acc_full[2], acc_free[2], done;
  uint32_t tmem;
};

// A warp's 32 rows of 64 bf16 to `map` at (x, y), through 4 KB of its own in the maps'
// 128-byte swizzle; v: this lane's row.
__device__ __forceinline__ void store_rows(const CUtensorMap* map, uint8_t* stage, int lane, int x, int y, const float* v) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the last rows have left
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    put8<1>(reinterpret_cast<__nv_bfloat16*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)), 0, v + 8 * j);
  ptx::fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) tma_store(map, stage, x, y);
}

// The same of 32 fp32 values.
__device__ __forceinline__ void store_rows_f32(const CUtensorMap* map, uint8_t* stage, int lane, int x, int y, const float* v) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<float4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  ptx::fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) tma_store(map, stage, x, y);
}

template <int PL, int G, int BN, int USE>
__global__ void __launch_bounds__(gemm_threads<PL>(), 1) ce_gemm_kernel(const __grid_constant__ CUtensorMap map_a,
                                                                  const __grid_constant__ CUtensorMap map_b,
                                                                  const __grid_constant__ CUtensorMap map_wa,
                                                                  const __grid_constant__ CUtensorMap map_wb,
                                                                  const __grid_constant__ CUtensorMap map_out,
                                                                  const __grid_constant__ GemmArgs a) {
  using C = GemmCfg<PL, G, BN>;
  constexpr int S = C::kStages;
  constexpr bool kConv = PL == 3 && USE != kWeight;   // the second operand comes from the warps that convert
  constexpr bool kBMN = USE != kStats && USE != kGrad;   // the second operand across its rows; the first too for the head's gradient
  extern __shared__ uint8_t raw_smem[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  GemmBars* bars = reinterpret_cast<GemmBars*>(sm + (size_t)S * C::kStage + C::kOut);
  const CePlan& pl = a.pl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = G == 2 ? blockIdx.x & 1 : 0, group = blockIdx.x / G, groups = gridDim.x / G;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(bars->full + s, 1 + (kConv ? kConvWarps : 0));
      ptx::mbar_init(bars->empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(bars->acc_full + b, 1);
      ptx::mbar_init(bars->acc_free + b, kEpiWarps * G);
    }
    ptx::mbar_init(&bars->done, 1);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&map_a);
    ptx::prefetch_tmap(&map_b);
  }
  if (warp == 2) tmem_alloc<G>(&bars->tmem);
  ptx::tc_fence_before();
  __syncthreads();
  sync_tile_ctas<G>();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem;
  griddep_wait();
  griddep_trigger();
  const int kept = *pl.kept;
  const Items<PL, G, BN, USE> items(a, kept, groups);
  const int n_items = items.n;

  if (warp == 0) {
    if (lane == 0) {   // ---------------------------------------------------- loads
      int it = 0;
      bool ok = true;
      for (int item = group; item < n_items && ok; item += groups) {
        int m0, n0, b0, b1;
        items.get(item, m0, n0, b0, b1);
        m0 += rank * kBM;
        n0 += rank * C::kOwnN;
        const bool w = items.weight(item);
        const CUtensorMap *ma = USE == kGrads && w ? &map_wa : &map_a, *mb = USE == kGrads && w ? &map_wb : &map_b;
        const int plane = pl.rows_pad;   // rows between an operand's planes
        const bool conv = kConv && !w;   // the head of fp32 tensors is not loaded here
        for (int kb = b0; kb < b1; ++kb, ++it) {
          const int s = it % S;
          if (it >= S && !ptx::mbar_wait(bars->empty + s, ((it / S) & 1) ^ 1, kBudget, pl.status)) {
            ok = false;
            break;
          }
          uint8_t* st = sm + (size_t)s * C::kStage;
          // the bytes of both CTAs count at the first one's barrier
          const uint32_t bar = G == 2 ? at_rank(bars->full + s, 0) : ptx::smem_u32(bars->full + s);
          if (rank == 0) ptx::mbar_arrive_expect_tx(bars->full + s, conv ? PL * C::kA : G * C::kStage);
#pragma unroll
          for (int p = 0; p < PL; ++p) {
            uint8_t* ta = st + p * C::kA;
            if (w) {
#pragma unroll
              for (int i = 0; i < kBM / 64; ++i) tma_tile<G>(ta + i * 8192, ma, bar, m0 + 64 * i, p * plane + kb * 64);
            } else {
              tma_tile<G>(ta, ma, bar, kb * 64, p * plane + m0);
            }
            if (conv) continue;
            uint8_t* tb = st + PL * C::kA + p * C::kB;
            if (kBMN) {
              const int row = w ? p * plane + kb * 64 : a.v0 + kb * 64;
#pragma unroll
              for (int i = 0; i < C::kOwnN / 64; ++i) tma_tile<G>(tb + i * 8192, mb, bar, n0 + 64 * i, row);
            } else {
              tma_tile<G>(tb, mb, bar, kb * 64, a.v0 + n0);
            }
          }
        }
      }
      // every load issued lands before the CTA can exit (the other CTA's wait for the
      // first one at the end)
      if (rank == 0)
        for (int j = max(0, it - S); j < it; ++j) ptx::mbar_wait(bars->full + j % S, (j / S) & 1, kBudget, nullptr);
    }
  } else if (warp == 1 && rank == 0) {   // --------------------------------- MMAs
    // The whole warp runs this, so that what it computes is uniform; one elected
    // lane issues each group of MMAs with the commits behind it.
    constexpr uint32_t kId = ptx::idesc_bf16_f32(C::kTM, C::kBN) | (kBMN ? 1u << 16 : 0u);
    constexpr uint32_t kb_ = k_step(kBMN);
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t p) {
      if (!__all_sync(0xffffffffu, try_wait_cluster(b, p))) {
        ok = ok && ptx::mbar_wait(b, p, kBudget, pl.status) && try_wait_cluster(b, p);
        ok = __all_sync(0xffffffffu, ok);
      }
      ptx::tc_fence_after();
      return ok;
    };
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t base = ptx::smem_u32(sm);
    int it = 0, seq = 0, small_seq = 0;
    for (int item = group; item < n_items && ok; item += groups) {
      int m0, n0, b0, b1;
      items.get(item, m0, n0, b0, b1);
      const bool w = items.weight(item);
      const uint32_t id = kId | (w ? 1u << 15 : 0u), ka = k_step(w);
      int sums = 0;
      for (int kb = b0; kb < b1 && ok; ++seq) {
        const int buf = seq & 1, use = seq >> 1;
        if (use >= 1 && !wait(bars->acc_free + buf, (use - 1) & 1)) break;
        const uint32_t d = tm + buf * C::kAccCols;
        // the small products' sum spans kSmallSums of the large one's; its two
        // accumulators lie behind the large one's two, and one is free again before
        // the last but one of the large one's is
        const uint32_t ds = tm + (2 + (small_seq & 1)) * C::kAccCols;
        const int end = min(kb + C::kSumBlocks, b1);
        uint32_t acc = 0;
        for (; kb < end; ++kb, ++it) {
          const int s = it % S;
          if (!wait(bars->full + s, (it / S) & 1)) break;
          const uint32_t da = desc_lo(base + s * C::kStage, w), db = desc_lo(base + s * C::kStage + PL * C::kA, kBMN);
          if (elect()) {
            if constexpr (PL == 1) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mma<G>(d, da + k * ka, db + k * kb_, id, acc | (k != 0));
            } else {
              // small products first: l h, h l, m m, m h, h m, then h h
              constexpr int qa[6] = {2, 0, 1, 1, 0, 0}, qb[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
              for (int q = 0; q < 6; ++q)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma<G>(q < 5 ? ds : d, da + (qa[q] * C::kA >> 4) + k * ka, db + (qb[q] * C::kB >> 4) + k * kb_, id,
                         q < 5 ? (acc | (sums != 0)) | (k != 0) | (q > 0) : acc | (k != 0));
            }
            commit<G>(bars->empty + s);
            if (kb + 1 == end) commit<G>(bars->acc_full + buf);
          }
          __syncwarp();
          acc = 1;
        }
        if (++sums == C::kSmallSums || kb == b1) sums = 0, ++small_seq;
      }
    }
    if (elect()) commit_own<G>(&bars->done);
    __syncwarp();
    ptx::mbar_wait(&bars->done, 0, kBudget, nullptr);   // what was issued ends before the CTAs do
  } else if (kConv && warp >= 4 + kEpiWarps) {   // ------------------------ the head's planes
    // A thread takes kPasses runs of eight values of a block: a run is 16 bytes of each
    // plane's row, in the 128-byte swizzle that a tensor map's load would give it.
    constexpr int kRunsRow = kBMN ? C::kBN / 8 : 8;           // runs in a row of the block
    constexpr int kRowsPass = 32 * kConvWarps / kRunsRow, kPasses = (kBMN ? 64 : C::kBN) / kRowsPass;
    static_assert(kRowsPass % 8 == 0 || PL != 3, "one swizzle a thread");
    const int t = threadIdx.x - 32 * (4 + kEpiWarps), run = t % kRunsRow, row0 = t / kRunsRow;
    struct Block {   // a K block of an item
      int item, n0, kb, end;
      bool more;
    };
    auto open = [&](Block& x) {   // the next item's first block, if there is one
      for (; x.item < n_items; x.item += groups) {
        int m0, b0;
        items.get(x.item, m0, x.n0, b0, x.end);
        x.kb = b0;
        if (b0 < x.end) return;
      }
      x.more = false;
    };
    auto next = [&](Block& x) {
      if (++x.kb < x.end) return;
      x.item += groups;
      open(x);
    };
    float4 buf[kPasses][2];   // of the block whose values are on their way
    Block cur{group, 0, 0, 0, true};
    open(cur);
    // where this thread's first run of the block lies, and how many of its rows there are
    const size_t step = (size_t)kRowsPass * pl.dim;
    const float* src = nullptr;
    int left = 0;
    auto aim = [&] {
      const int v = kBMN ? cur.kb * 64 + row0 : cur.n0 + row0, d = 8 * run + (kBMN ? cur.n0 : cur.kb * 64);
      left = cur.more && !items.weight(cur.item) && d < pl.dim ? a.cols - v : 0;
      src = static_cast<const float*>(a.weight) + (size_t)(a.v0 + v) * pl.dim + d;
    };
    auto fetch = [&](int p) {
      const bool in = p * kRowsPass < left;
      const float4* x = reinterpret_cast<const float4*>(src + p * step);
      buf[p][0] = in ? __ldg(x) : make_float4(0.f, 0.f, 0.f, 0.f);
      buf[p][1] = in ? __ldg(x + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    uint8_t* const planes = sm + PL * C::kA + row0 * 128 + (((run & 7) ^ (row0 & 7)) << 4) + (kBMN ? (run >> 3) * 8192 : 0);
    aim();
#pragma unroll
    for (int p = 0; p < kPasses; ++p) fetch(p);
    for (int it = 0; cur.more; ++it) {
      const int s = it % S;
      const bool skip = items.weight(cur.item);   // (that block's second operand comes by TMA)
      next(cur);
      aim();
      if (it >= S && !__all_sync(0xffffffffu, ptx::mbar_wait(bars->empty + s, ((it / S) & 1) ^ 1, kBudget, pl.status))) break;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        if (!skip) {   // (rows 8 apart have the same swizzle)
          const float v[8] = {buf[p][0].x, buf[p][0].y, buf[p][0].z, buf[p][0].w, buf[p][1].x, buf[p][1].y, buf[p][1].z, buf[p][1].w};
          put8<PL>(reinterpret_cast<__nv_bfloat16*>(planes + (size_t)s * C::kStage + p * kRowsPass * 128), C::kB / 2, v);
        }
        fetch(p);
      }
      ptx::fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars->full + s);
    }
  } else if (warp >= 4 && warp < 4 + kEpiWarps) {   // ---------------------- sums
    constexpr int NC = C::kNC;
    const int half = (warp - 4) >> 2, lane_row = 32 * (warp & 3) + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const int c_half = half * NC;
    uint8_t* stage = sm + (size_t)S * C::kStage + (warp - 4) * 4096;
    const uint32_t free0 = G == 2 ? at_rank(bars->acc_free, 0) : ptx::smem_u32(bars->acc_free);
    int seq = 0, small_seq = 0;
    bool ok = true;
    // what a row needs at the end of its tile, loaded while the tile before is at work
    struct Row {
      int target;
      float2 l2;
      float gain;
    };
    auto row_of_item = [&](int item) {
      Row r{-1, make_float2(0.f, 0.f), 0.f};
      if ((USE == kStats || USE == kGrad) && item < n_items) {
        int m0, n0, b0, b1;
        items.get(item, m0, n0, b0, b1);
        const int row = m0 + rank * kBM + lane_row;
        if (row < kept) {
          r.target = pl.target[row];
          if (USE == kGrad) {
            r.l2 = pl.lse2[row];
            r.gain = pl.gain[row];
          }
        }
      }
      return r;
    };
    Row next = row_of_item(group);
    for (int item = group; item < n_items && ok; item += groups) {
      int m0, n0, b0, b1;
      items.get(item, m0, n0, b0, b1);
      m0 += rank * kBM;
      const int row = m0 + lane_row;   // (a vocabulary row of the piece for the head's gradient)
      const bool in = (USE == kStats || USE == kGrad) && row < kept;
      const int target = next.target;
      const float2 l2 = next.l2;
      const float gain = next.gain;
      next = row_of_item(item + groups);
      float acc[NC];
      if (b0 == b1) {
#pragma unroll
        for (int j = 0; j < NC; ++j) acc[j] = 0.f;
      }
      int sums = 0;
      for (int kb = b0; kb < b1; kb += C::kSumBlocks, ++seq) {
        const int buf = seq & 1;
        if (!ptx::mbar_wait(bars->acc_full + buf, (seq >> 1) & 1, kBudget, pl.status)) ok = false;
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        auto drain = [&](uint32_t at) {
#pragma unroll
          for (int j0 = 0; j0 < NC; j0 += 16) {
            float v[16];
            ptx::tmem_ld16(at + j0, v);
#pragma unroll
            for (int j = 0; j < 16; j += 2)
              split2(add2(two(acc[j0 + j], acc[j0 + j + 1]), two(v[j], v[j + 1])), acc[j0 + j], acc[j0 + j + 1]);
          }
        };
        const uint32_t at = tmem + lanes + buf * C::kAccCols + c_half;
        if (kb == b0) {   // the first sum as it is
#pragma unroll
          for (int j0 = 0; j0 < NC; j0 += 32) tmem_load32(at + j0, acc + j0);
          tmem_loaded<NC>(acc);
        } else {
          drain(at);
        }
        if (PL == 3 && (++sums == C::kSmallSums || kb + C::kSumBlocks >= b1)) {
          drain(tmem + lanes + (2 + (small_seq & 1)) * C::kAccCols + c_half);
          sums = 0;
          ++small_seq;
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(free0 + buf * 8);
      }
      if (!ok) break;
      const int col = n0 + c_half;     // within the piece, or the dim
      if constexpr (USE == kStats) {
        const int left = a.cols - col;                     // columns that there are
        const int tgt = target - a.v0 - col;
        const uint64_t scale = two(a.scale2, a.scale2);
#pragma unroll
        for (int j = 0; j < NC; j += 2) split2(mul2(two(acc[j], acc[j + 1]), scale), acc[j], acc[j + 1]);
        if (left < NC) {
#pragma unroll
          for (int j = 0; j < NC; ++j)
            if (j >= left) acc[j] = -INFINITY;
        }
        if (__any_sync(0xffffffffu, in && (unsigned)tgt < (unsigned)NC)) {
#pragma unroll
          for (int j = 0; j < NC; ++j)
            if (in && j == tgt) pl.picked[row] = acc[j];
        }
        float m = -INFINITY, s = 0.f;
#pragma unroll
        for (int j0 = 0; j0 < NC; j0 += 32) {
          float gm = acc[j0];
#pragma unroll
          for (int j = j0 + 1; j < j0 + 32; ++j) gm = fmaxf(gm, acc[j]);
          const float nm = fmaxf(m, gm), ref = nm == -INFINITY ? 0.f : nm;
          s *= ex2(m - ref);
          const uint64_t less = two(-ref, -ref);
          float part[2] = {0.f, 0.f};
#pragma unroll
          for (int j = j0; j < j0 + 32; j += 2) {
            float x, y;
            split2(add2(two(acc[j], acc[j + 1]), less), x, y);
            part[0] += ex2(x);
            part[1] += ex2(y);
          }
          s += part[0] + part[1];
          m = nm;
        }
        if (in) pl.part[(size_t)(2 * (n0 / C::kBN) + half) * pl.rows_pad + row] = make_float2(m, s);
      } else if constexpr (USE == kGrad) {
        // 64 columns at a time: one half's values are made while the other's leave
#pragma unroll
        for (int h = 0; h < NC; h += 64) {
          float* g = acc + h;
          const int left = in ? a.cols - col - h : 0, tgt = target - a.v0 - col - h;
          const uint64_t scale = two(a.scale2, a.scale2), less = two(-l2.x, -l2.x), times = two(gain, gain);
#pragma unroll
          for (int j = 0; j < 64; j += 2) {
            const uint64_t z = two(g[j], g[j + 1]);
            uint64_t e = fma2(z, scale, less);
            if (PL == 3) e = fma2(z, two(a.scale2_lo, a.scale2_lo), add2(e, two(-l2.y, -l2.y)));
            split2(e, g[j], g[j + 1]);
            g[j] = ex2(g[j]);
            g[j + 1] = ex2(g[j + 1]);
          }
#pragma unroll
          for (int j = 0; j < 64; j += 2) split2(mul2(two(g[j], g[j + 1]), times), g[j], g[j + 1]);
          if (__any_sync(0xffffffffu, (unsigned)tgt < 64u)) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (j == tgt) {
                g[j] -= gain;
                // the target's value is often the row's largest by far: what its rounding
                // leaves is made good in the hidden states' gradient
                if (PL == 1) pl.rest[row] = g[j] - __bfloat162float(__float2bfloat16_rn(g[j]));
              }
          }
          if (__any_sync(0xffffffffu, left < 64)) {   // behind the head's last row, and rows behind the kept ones
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (j >= left) g[j] = 0.f;
          }
#pragma unroll
          for (int p = 0; p < PL; ++p) {   // a plane, then what it leaves
            store_rows(&map_out, stage, lane, col + h, p * pl.rows_pad + m0 + 32 * (warp & 3), g);
            if (p + 1 < PL) {
#pragma unroll
              for (int j = 0; j < 64; ++j) g[j] -= __bfloat162float(__float2bfloat16_rn(g[j]));
            }
          }
        }
      } else if (items.weight(item)) {
        // (rows behind the head's last and columns behind the dim are cut off by the map)
        constexpr int kCols = PL == 1 ? 64 : 32;
#pragma unroll
        for (int j0 = 0; j0 < NC; j0 += kCols)
          if (m0 + 32 * (warp & 3) < a.cols && col + j0 < pl.dim) {
            if constexpr (PL == 1) store_rows(&map_out, stage, lane, col + j0, a.v0 + m0 + 32 * (warp & 3), acc + j0);
            else store_rows_f32(&map_out, stage, lane, col + j0, a.v0 + m0 + 32 * (warp & 3), acc + j0);
          }
      } else if (pl.direct) {   // the one piece of a small vocabulary: to the caller's rows
        if (row < kept) {
          using T = typename Tensor<PL>::T;
          T* out = static_cast<T*>(a.d_hidden) + pl.row_of[row] * a.d_row_stride + col;
          const bool vec = rows_vec(static_cast<T*>(a.d_hidden), a.d_row_stride);
          const T* w = static_cast<const T*>(a.weight) + (size_t)pl.target[row] * pl.dim + col;
          const float rest = PL == 1 ? pl.rest[row] : 0.f;
          const int left = pl.dim - col;   // a multiple of 8
#pragma unroll
          for (int j = 0; j < NC; j += 8)
            if (j < left) {
              if (PL == 1) add_rest(w + j, rest, acc + j);
              set8(out + j, vec, acc + j);
            }
        }
      } else {
        // whole tiles to their place, parts of a tile to a tile of their own; a piece
        // adds to what the pieces before it left (each value once a launch: the order
        // of the additions is fixed)
        const bool part = item >= items.whole;
        float* out = part ? pl.tail + ((size_t)(item - items.whole) * C::kTM + rank * kBM + lane_row) * C::kBN + c_half
                          : pl.acc + (size_t)row * pl.dim_pad + col;
        const int left = part ? NC : pl.dim_pad - col;
        if (a.first) {
#pragma unroll
          for (int j = 0; j < NC; j += 4)
            if (j < left) *reinterpret_cast<float4*>(out + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < NC; j += 4)
            if (j < left) red_add4(out + j, acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  sync_tile_ctas<G>();   // neither CTA leaves while the other's MMAs or arrivals may reach it
  if (warp == 2) {
    ptx::tc_fence_after();
    tmem_free<G>(tmem);
  }
}

// ---------------------------------------------------------------- ends
// A row's pairs merged: lse = ln2 (M + log2 S), and the loss from the difference of
// the exponents, which is exact where the target has the largest.
// A CTA takes ROWS rows, its threads a share of the pairs each: 32 rows' pairs lie in
// 256 bytes, but few rows need more CTAs.  Latency: 6 us for 15 rows of 1,188 pairs and for
// 777 of 252 (32 rows a CTA for the former: 14.7).
constexpr int kMergeThreads = 512;

template <int ROWS>
__global__ void __launch_bounds__(kMergeThreads) ce_merge_kernel(CePlan pl, int parts, float* loss, float* lse) {
  griddep_wait();
  griddep_trigger();
  constexpr int kWarps = kMergeThreads / 32, kStep = kMergeThreads / ROWS, U = 4;
  __shared__ float2 sh[kWarps][ROWS];
  const int tid = threadIdx.x, warp = tid >> 5, r0 = blockIdx.x * ROWS, r = r0 + tid % ROWS, kept = *pl.kept;
  if (r0 >= kept) return;
  float m = -INFINITY, s = 0.f;
  auto add = [&](float2 v) {
    const float nm = fmaxf(m, v.x), ref = nm == -INFINITY ? 0.f : nm;
    s = s * ex2(m - ref) + v.y * ex2(v.x - ref);
    m = nm;
  };
  if (r < kept)
    for (int p = tid / ROWS; p < parts; p += U * kStep) {
      float2 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = p + u * kStep < parts ? pl.part[(size_t)(p + u * kStep) * pl.rows_pad + r] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int u = 0; u < U; ++u) add(v[u]);
    }
#pragma unroll
  for (int o = ROWS; o < 32; o *= 2) {   // the warp's shares of a row
    const float2 v = make_float2(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o));
    add(v);
  }
  if ((tid & 31) < ROWS) sh[warp][tid & 31] = make_float2(m, s);
  __syncthreads();
  if (tid < ROWS && r < kept) {
    for (int w = 1; w < kWarps; ++w) add(sh[w][tid]);
    const float l2 = log2f(s);
    const int to = pl.row_of[r];
    lse[to] = kLn2 * (m + l2);
    loss[to] = kLn2 * ((m - pl.picked[r]) + l2);
  }
}

// The hidden states' gradient to the caller's rows, the parts of a cut tile added in
// order.  HBM and L2: 34 us for 4,096 x 4,096, 5 for 300 x 256.
constexpr int kFinishThreads = 256;

template <typename T, int PL, int G, int BN>
__global__ void __launch_bounds__(kFinishThreads) ce_finish_hidden_kernel(CePlan pl, const T* weight, T* d_hidden, int64_t stride, int groups_of_ctas) {
  griddep_wait();
  griddep_trigger();
  using C = GemmCfg<PL, G, BN>;
  const int kept = *pl.kept;
  const int m_tiles = (kept + C::kTM - 1) / C::kTM, tiles = m_tiles * ((pl.dim + C::kBN - 1) / C::kBN), parts = pl.kept[1];
  const int rest = parts > 1 ? tiles % groups_of_ctas : 0, whole = tiles - rest;
  const bool vec = rows_vec(d_hidden, stride);
  const size_t step = (size_t)rest * C::kTM * C::kBN;
  for (int r = blockIdx.x; r < kept; r += gridDim.x) {
    T* out = d_hidden + pl.row_of[r] * stride;
    const T* w = weight + (size_t)pl.target[r] * pl.dim;
    const float rest_r = PL == 1 ? pl.rest[r] : 0.f;
    for (int c = threadIdx.x * 8; c < pl.dim; c += kFinishThreads * 8) {
      const int tile = c / C::kBN * m_tiles + r / C::kTM;
      float sum[8];
      if (tile < whole) {
        get8(pl.acc + (size_t)r * pl.dim_pad + c, true, sum);
      } else {
        const float* src = pl.tail + ((size_t)(tile - whole) * C::kTM + r % C::kTM) * C::kBN + c % C::kBN;
        get8(src, true, sum);
        for (int p = 1; p < parts; p += 4) {
          float v[4][8];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (p + u < parts) get8(src + (p + u) * step, true, v[u]);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (p + u < parts) {
#pragma unroll
              for (int j = 0; j < 8; ++j) sum[j] += v[u][j];
            }
        }
      }
      if (PL == 1) add_rest(w + c, rest_r, sum);
      set8(out + c, vec, sum);
    }
  }
}

// ---------------------------------------------------------------- host side
template <int PL, int G, int BN>
cudaError_t prepare() {
  for (auto kernel : {ce_gemm_kernel<PL, G, BN, kStats>, ce_gemm_kernel<PL, G, BN, kGrad>, ce_gemm_kernel<PL, G, BN, kHidden>,
                      ce_gemm_kernel<PL, G, BN, kWeight>, ce_gemm_kernel<PL, G, BN, kGrads>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)GemmCfg<PL, G, BN>::kBytes);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int gemm_groups(int ctas, int sms) { return std::max(1, sms / ctas); }

template <int PL, int G, int BN, int USE>
cudaError_t gemm(const GemmArgs& a, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& wa, const CUtensorMap& wb,
                 const CUtensorMap& mo, int sms, int* launches, cudaStream_t s) {
  ++*launches;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(G * gemm_groups(G, sms));
  cfg.blockDim = dim3(gemm_threads<PL>());
  cfg.dynamicSmemBytes = GemmCfg<PL, G, BN>::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (G > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = G;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, ce_gemm_kernel<PL, G, BN, USE>, ma, mb, wa, wb, mo, a);
}

struct Scale {
  float hi, lo;
};
Scale scale_of(float temperature) {
  const double s = 1.4426950408889634074 / (double)temperature;
  Scale r;
  r.hi = (float)s;
  r.lo = (float)(s - (double)r.hi);
  return r;
}

// Rows a CTA of the first kernel takes: each counts all targets, so no more than 1,024 CTAs.
int gather_rows(int rows) { return std::max(8, (rows + 1023) / 1024); }
// (and at least as many as fill a tile's padding a row a warp)
constexpr int kTilePad = 2 * kBM / (kGatherThreads / 32);
template <typename T, int PL, int G, int BN>
cudaError_t forward(const CePlan& pl, const CeTensors& t, int sms, int* launches, cudaStream_t s) {
  using C = GemmCfg<PL, G, BN>;
  const int per = gather_rows(pl.rows), ctas = std::max((pl.rows + per - 1) / per, kTilePad);
  cudaError_t e = launch_pdl(ce_gather_kernel<T, PL, false>, dim3(ctas), dim3(kGatherThreads), 0, s,
                             pl, t, per, gemm_groups(G, sms));
  ++*launches;
  if (e != cudaSuccess) return e;
  CUtensorMap mh, mw;
  if (!encode_activation_map(&mh, pl.h, pl.dim_pad, PL * pl.rows_pad, pl.dim_pad, kBM)) return cudaErrorInvalidValue;
  mw = mh;
  if (PL == 1 && !encode_activation_map(&mw, t.weight, pl.dim, pl.vocab, pl.dim, C::kOwnN)) return cudaErrorInvalidValue;
  GemmArgs a{};
  a.pl = pl;
  const Scale sc = scale_of(t.temperature);
  a.scale2 = sc.hi;
  a.scale2_lo = sc.lo;
  a.weight = t.weight;
  a.cols = pl.vocab;
  e = gemm<PL, G, BN, kStats>(a, mh, mw, mh, mw, mw, sms, launches, s);
  if (e != cudaSuccess) return e;
  const int parts = 2 * ((pl.vocab + BN - 1) / BN);
  ++*launches;
  const bool few = pl.rows <= 4 * sms;
  return launch_pdl(few ? ce_merge_kernel<4> : ce_merge_kernel<32>, dim3(few ? (pl.rows + 3) / 4 : (pl.rows + 31) / 32),
                    dim3(kMergeThreads), 0, s, pl, parts, t.loss, t.lse);
}

template <typename T, int PL, int G, int BN>
cudaError_t backward(const CePlan& pl, const CeTensors& t, int sms, int* launches, cudaStream_t s) {
  using C = GemmCfg<PL, G, BN>;
  const int per = gather_rows(pl.rows), ctas = std::max((pl.rows + per - 1) / per, kTilePad);
  cudaError_t e = launch_pdl(ce_gather_kernel<T, PL, true>, dim3(ctas), dim3(kGatherThreads), 0, s,
                             pl, t, per, gemm_groups(G, sms));
  ++*launches;
  if (e != cudaSuccess) return e;
  // operands with the product's K along their rows (boxes of 64 x rows of the tile) or across them (64 x 64)
  CUtensorMap h_k, h_mn, w_k, w_mn, g_k, g_mn, g_out, dw_out{};
  if (!encode_activation_map(&h_k, pl.h, pl.dim_pad, PL * pl.rows_pad, pl.dim_pad, kBM) ||
      !encode_activation_map(&h_mn, pl.h, pl.dim_pad, PL * pl.rows_pad, pl.dim_pad, 64) ||
      !encode_activation_map(&g_k, pl.g, pl.piece, PL * pl.rows_pad, pl.piece, kBM) ||
      !encode_activation_map(&g_mn, pl.g, pl.piece, PL * pl.rows_pad, pl.piece, 64) ||
      !encode_activation_map(&g_out, pl.g, pl.piece, PL * pl.rows_pad, pl.piece, 32) ||
      (t.d_weight && !(PL == 1 ? encode_activation_map(&dw_out, t.d_weight, pl.dim, pl.vocab, pl.dim, 32)
                               : encode_f32_map(&dw_out, t.d_weight, pl.dim, pl.vocab, 32))))
    return cudaErrorInvalidValue;
  w_k = w_mn = h_k;   // (fp32: not read)
  if (PL == 1 && (!encode_activation_map(&w_k, t.weight, pl.dim, pl.vocab, pl.dim, C::kOwnN) ||
                  !encode_activation_map(&w_mn, t.weight, pl.dim, pl.vocab, pl.dim, 64)))
    return cudaErrorInvalidValue;
  GemmArgs a{};
  a.pl = pl;
  const Scale sc = scale_of(t.temperature);
  a.scale2 = sc.hi;
  a.scale2_lo = sc.lo;
  a.weight = t.weight;
  a.d_hidden = t.d_hidden;
  a.d_row_stride = t.d_row_stride;
  // (the tiles of a piece's two gradients)
  const long long tiles = (long long)(pl.rows_pad / pl.tile + (pl.piece + pl.tile - 1) / pl.tile) * ((pl.dim + BN - 1) / BN);
  const bool both = t.d_hidden && t.d_weight && tiles <= 4LL * gemm_groups(G, sms);
  for (int v0 = 0; v0 < pl.vocab; v0 += pl.piece) {
    a.v0 = v0;
    a.cols = std::min(pl.piece, pl.vocab - v0);
    a.first = v0 == 0;
    if ((e = gemm<PL, G, BN, kGrad>(a, h_k, w_k, h_k, w_k, g_out, sms, launches, s)) != cudaSuccess) return e;
    if (both) {
      if ((e = gemm<PL, G, BN, kGrads>(a, g_k, w_mn, g_mn, h_mn, dw_out, sms, launches, s)) != cudaSuccess) return e;
      continue;
    }
    if (t.d_hidden && (e = gemm<PL, G, BN, kHidden>(a, g_k, w_mn, g_k, w_mn, g_out, sms, launches, s)) != cudaSuccess) return e;
    if (t.d_weight && (e = gemm<PL, G, BN, kWeight>(a, g_mn, h_mn, g_mn, h_mn, dw_out, sms, launches, s)) != cudaSuccess) return e;
  }
  if (!t.d_hidden || pl.direct) return cudaSuccess;
  ++*launches;
  return launch_pdl(ce_finish_hidden_kernel<T, PL, G, BN>, dim3(std::min(pl.rows, sms * 64)), dim3(kFinishThreads), 0, s, pl,
                    static_cast<const T*>(t.weight), static_cast<T*>(t.d_hidden), t.d_row_stride, gemm_groups(G, sms));
}

}  // namespace

CePlan ce_plan(void* ws, int rows, int dim, int vocab, bool f32, bool backward, bool want_hidden, int sms) {
  CePlan pl{};
  pl.rows = rows;
  pl.dim = dim;
  pl.vocab = vocab;
  pl.planes = f32 ? 3 : 1;
  // Tiles.  A pair of CTAs shares 256 x 256, unless there is one CTA's worth of rows
  // (the second would only hold up half the loads: 15 rows of 4,096 against 151,936 in
  // 237 us, alone 198); where tiles of 128 x 128 fit one wave their K, the time of such
  // a call, takes half as long a block.
  const long long tiles128 = (long long)((rows + kBM - 1) / kBM) * ((vocab + 127) / 128);
  const bool small = !f32 && tiles128 <= sms;
  pl.bn = f32 || small ? 128 : 256;
  pl.ctas = f32 || small || rows <= kBM || sms < 2 ? 1 : 2;
  pl.tile = kBM * pl.ctas;
  pl.rows_pad = (rows + pl.tile - 1) / pl.tile * pl.tile;
  pl.dim_pad = (dim + 63) / 64 * 64;
  const int bn = pl.bn;
  // pieces of equal size, as few as the limit allows
  const size_t column = 2 * (size_t)pl.planes * pl.rows_pad;
  const long long limit = std::max<long long>(256, (long long)(kPieceBytes / column) / 256 * 256);
  const long long all = ((long long)vocab + 255) / 256 * 256;
  if (!backward) {
    pl.piece = (int)all;   // nothing is stored
  } else {
    const long long n = (all + limit - 1) / limit;
    pl.piece = (int)((all / 256 + n - 1) / n * 256);
  }
  char* p = static_cast<char*>(ws);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* r = p ? p + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return r;
  };
  int32_t* head = reinterpret_cast<int32_t*>(take(256));
  pl.status = head;
  pl.kept = head ? head + 1 : nullptr;
  const size_t R = pl.rows_pad;
  pl.row_of = reinterpret_cast<int32_t*>(take(4 * R));
  pl.target = reinterpret_cast<int32_t*>(take(4 * R));
  pl.h = reinterpret_cast<__nv_bfloat16*>(take(2 * pl.planes * R * pl.dim_pad));
  if (!backward) {
    pl.part = reinterpret_cast<float2*>(take(sizeof(float2) * 2 * (size_t)((vocab + bn - 1) / bn) * R));
    pl.picked = reinterpret_cast<float*>(take(4 * R));
  } else {
    pl.lse2 = reinterpret_cast<float2*>(take(8 * R));
    pl.gain = reinterpret_cast<float*>(take(4 * R));
    pl.rest = reinterpret_cast<float*>(take(4 * R));
    pl.g = reinterpret_cast<__nv_bfloat16*>(take(2 * pl.planes * R * pl.piece));
    // a small vocabulary's K is short: no tile is cut, and the tiles go to the caller's rows
    pl.direct = pl.piece >= vocab && pl.piece <= kDirectPiece;
    if (want_hidden && !pl.direct) {
      pl.acc = reinterpret_cast<float*>(take(4 * R * pl.dim_pad));
      pl.tail = reinterpret_cast<float*>(take(4 * (size_t)kTailWaves * sms * kBM * bn));
    }
  }
  pl.bytes = off;
  return pl;
}

cudaError_t ce_prepare_f32() { return prepare<3, 1, 128>(); }
cudaError_t ce_prepare_bf16() {
  for (cudaError_t e : {prepare<1, 1, 128>(), prepare<1, 1, 256>(), prepare<1, 2, 256>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

cudaError_t ce_forward(const CePlan& pl, const CeTensors& t, int sms, int* launches, cudaStream_t s) {
  *launches = 0;
  if (pl.planes == 3) return forward<float, 3, 1, 128>(pl, t, sms, launches, s);
  if (pl.bn == 128) return forward<__nv_bfloat16, 1, 1, 128>(pl, t, sms, launches, s);
  return pl.ctas == 2 ? forward<__nv_bfloat16, 1, 2, 256>(pl, t, sms, launches, s)
                      : forward<__nv_bfloat16, 1, 1, 256>(pl, t, sms, launches, s);
}

cudaError_t ce_backward(const CePlan& pl, const CeTensors& t, int sms, int* launches, cudaStream_t s) {
  *launches = 0;
  if (pl.planes == 3) return backward<float, 3, 1, 128>(pl, t, sms, launches, s);
  if (pl.bn == 128) return backward<__nv_bfloat16, 1, 1, 128>(pl, t, sms, launches, s);
  return pl.ctas == 2 ? backward<__nv_bfloat16, 1, 2, 256>(pl, t, sms, launches, s)
                      : backward<__nv_bfloat16, 1, 1, 256>(pl, t, sms, launches, s);
}

}  // namespace dflash
