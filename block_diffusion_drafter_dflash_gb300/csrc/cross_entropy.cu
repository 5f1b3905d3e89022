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
// One GEMM kernel with four uses:
//   stats    z of a tile of 128 rows x 256 vocabulary columns, reduced in registers
//            to a (maximum, sum) pair a row and half tile, and the target's z
//   grad     z again, turned into G: a piece of it is stored, rounded to bf16
//   hidden   dH += G W over a piece (W read with its vocabulary axis along K)
//   weight   dW = G' H of a piece's rows of the head (both along the rows)
// A piece is as many columns as keep G within kPieceBytes.
//
// A thread loads tiles by TMA into a ring, one warp issues the MMAs, eight warps
// read the sums.  The tensor cores' fp32 sums truncate (by 2e-8 of the sum a step
// of 16, to one side), which over a dim of 4,096 would put the loss off by 3e-6 of
// itself; so a sum ends after kSumBlocks blocks of 64 and the eight warps add it to
// fp32 registers, two accumulators taking turns.
//
// fp32 tensors enter as three bf16 planes each (x = h + m + l, 24 bits), every
// product as six (h h, h m, m h, m m, h l, l h; what is left out is below 2^-24),
// the five small ones with a sum of their own.
#include <cuda.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "cross_entropy.cuh"
#include "gemm.cuh"
#include "ptx.cuh"

namespace dflash {
namespace {

constexpr int kBM = 128;                 // rows of an output tile
constexpr int kSumBlocks = 8;            // K blocks of 64 that one sum of the tensor cores spans
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = 128 + 32 * kEpiWarps;
constexpr long long kBudget = 400000000LL;
constexpr float kLn2 = 0.6931471805599453f;
constexpr size_t kPieceBytes = size_t(192) << 20;

enum Use { kStats, kGrad, kHidden, kWeight };

template <int PL>
struct GemmCfg {
  static constexpr int kBN = PL == 1 ? 256 : 128;
  static constexpr int kA = kBM * 128, kB = kBN * 128;     // bytes of a K block of 64
  static constexpr int kStage = PL * (kA + kB);
  static constexpr int kStages = PL == 1 ? 4 : 2;
  static constexpr int kAccCols = PL == 1 ? kBN : 2 * kBN; // tensor-memory columns of one accumulator (three planes: the small products' sum behind the large one's)
  static constexpr int kNC = kBN / 2;                      // columns of an epilogue thread
  static constexpr size_t kBytes = 1024 + (size_t)kStages * kStage + 256;
  static_assert(2 * kAccCols == 512, "two accumulators fill tensor memory");
};

struct GemmArgs {
  CePlan pl;
  int v0, cols;          // the piece's first vocabulary column, how many there are
  int first;             // hidden: the sums start here
  int part0;             // stats: the piece's first pair
  float scale2, scale2_lo;   // log2(e) / T and its rounding residual
  void* d_weight;
  int f32_out;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- planes
// x as one bf16, or as three whose sum has all its 24 bits.
template <int PL>
__device__ __forceinline__ void split_planes(float x, __nv_bfloat16* p) {
  p[0] = __float2bfloat16_rn(x);
  if constexpr (PL == 3) {
    if (__hisinf(p[0]) && !isinf(x)) p[0] = __float2bfloat16_rz(x);
    x -= __bfloat162float(p[0]);
    p[1] = __float2bfloat16_rn(x);
    p[2] = __float2bfloat16_rn(x - __bfloat162float(p[1]));
  }
}
__device__ __forceinline__ uint32_t pack2(__nv_bfloat16 a, __nv_bfloat16 b) {
  return (uint32_t)__bfloat16_as_ushort(a) | (uint32_t)__bfloat16_as_ushort(b) << 16;
}
// Eight values as planes `stride` elements apart, 16 bytes each.
template <int PL>
__device__ __forceinline__ void put8(__nv_bfloat16* dst, size_t stride, const float* v) {
  __nv_bfloat16 p[8][PL];
#pragma unroll
  for (int j = 0; j < 8; ++j) split_planes<PL>(v[j], p[j]);
#pragma unroll
  for (int k = 0; k < PL; ++k)
    *reinterpret_cast<uint4*>(dst + k * stride) =
        make_uint4(pack2(p[0][k], p[1][k]), pack2(p[2][k], p[3][k]), pack2(p[4][k], p[5][k]), pack2(p[6][k], p[7][k]));
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
template <typename T>
__device__ __forceinline__ bool rows_vec(const T* p, int64_t stride) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(stride * (int64_t)sizeof(T))) & 15) == 0;
}

// ---------------------------------------------------------------- rows that count
// Kept rows in their order: where each came from, its target and statistics, and
// its hidden state as planes.  Every CTA counts the kept rows before its own.
// Ignored rows get their results here: loss and lse 0, or a gradient of zeros.
constexpr int kGatherThreads = 256;

template <typename T, int PL, bool BWD>
__global__ void __launch_bounds__(kGatherThreads) ce_gather_kernel(CePlan pl, CeTensors t, int per) {
  griddep_wait();
  griddep_trigger();
  __shared__ int s_before, s_total, s_warp[kGatherThreads / 32], s_list[kGatherThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_before = s_total = 0;
  __syncthreads();
  const int r0 = blockIdx.x * per, r1 = min(r0 + per, pl.rows);
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
  if (blockIdx.x == 0 && tid == 0) {
    *pl.status = 0;
    *pl.kept = total;
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
        for (int c = lane * 8; c < pl.dim_pad; c += 256) {
          float v[8] = {};
          if (c < pl.dim) get8(src + c, vec, v);
          put8<PL>(dst + c, plane, v);
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
  const int end = min((total + kBM - 1) / kBM * kBM, pl.rows_pad);
  for (int p = total + blockIdx.x * (kGatherThreads / 32) + warp; p < end; p += gridDim.x * (kGatherThreads / 32)) {
    __nv_bfloat16* dst = pl.h + (size_t)p * pl.dim_pad;
    for (int c = lane * 8; c < pl.dim_pad; c += 256) put8<PL>(dst + c, plane, zero);
  }
}

// A piece of an fp32 head as three planes, zero behind its last row and column.
__global__ void __launch_bounds__(256) ce_split_weight_kernel(CePlan pl, const float* w, int v0) {
  griddep_wait();
  griddep_trigger();
  const int groups = pl.dim_pad / 8;
  const bool vec = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
  const size_t plane = (size_t)pl.piece * pl.dim_pad;
  const long long n = (long long)pl.piece * groups;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const int r = (int)(i / groups), c = (int)(i - (long long)r * groups) * 8;
    float v[8] = {};
    if (v0 + r < pl.vocab && c < pl.dim) get8(w + (size_t)(v0 + r) * pl.dim + c, vec, v);
    put8<3>(pl.w + (size_t)r * pl.dim_pad + c, plane, v);
  }
}

// ---------------------------------------------------------------- tensor-core pieces
// High word of every shared-memory descriptor: 128-byte swizzle, 8 rows are 1024 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// K-major: a row's 64 values run along K.  MN-major: they run along M or N, the
// rows along K, and the tile of the next 64 is 64 rows further.
template <bool MN>
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) {
  return (addr >> 4) | ((MN ? 8192u >> 4 : 1u) << 16);
}
template <bool MN>
__host__ __device__ constexpr uint32_t k_step() { return MN ? 16 * 128 >> 4 : 32 >> 4; }   // 16 along K

__device__ __forceinline__ bool elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_tile(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                   ptx::smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(x), "r"(y)
               : "memory");
}

// Items of a launch: output tiles (with a share of K for the hidden states' gradient).
template <int PL, int USE>
struct Items {
  int m_tiles, n_tiles, splits, blocks;   // blocks: K blocks of 64
  __device__ __forceinline__ Items(const GemmArgs& a, int kept) {
    using C = GemmCfg<PL>;
    const CePlan& pl = a.pl;
    splits = 1;
    if (USE == kWeight) {
      m_tiles = (a.cols + kBM - 1) / kBM;
      n_tiles = (pl.dim + C::kBN - 1) / C::kBN;
      blocks = (kept + 63) / 64;
    } else {
      m_tiles = (kept + kBM - 1) / kBM;
      if (USE == kHidden) {
        n_tiles = (pl.dim + C::kBN - 1) / C::kBN;
        blocks = (a.cols + 63) / 64;
        splits = pl.splits;
      } else {
        n_tiles = (a.cols + C::kBN - 1) / C::kBN;
        blocks = pl.dim_pad / 64;
      }
    }
  }
  __device__ __forceinline__ int count() const { return m_tiles * n_tiles * splits; }
  // first row and column of the item's tile, and its K blocks
  __device__ __forceinline__ void get(int item, int& m0, int& n0, int& b0, int& b1) const {
    int mt, nt, sp = 0;
    if (USE == kWeight) {   // along a row of tiles: G's columns stay in L2
      nt = item % n_tiles;
      mt = item / n_tiles;
    } else {
      mt = item % m_tiles;
      nt = item / m_tiles;
      if (USE == kHidden) {
        sp = nt / n_tiles;
        nt -= sp * n_tiles;
      }
    }
    m0 = mt * kBM;
    n0 = nt * GemmCfg<PL>::kBN;
    b0 = (int)((long long)blocks * sp / splits);
    b1 = (int)((long long)blocks * (sp + 1) / splits);
  }
  __device__ __forceinline__ int split_of(int item) const { return item / (m_tiles * n_tiles); }
};

struct GemmBars {
  uint64_t full[4], empty[4], acc_full[2], acc_free[2], done;
  uint32_t tmem;
};

template <int PL, int USE>
__global__ void __launch_bounds__(kGemmThreads, 1) ce_gemm_kernel(const __grid_constant__ CUtensorMap map_a,
                                                                  const __grid_constant__ CUtensorMap map_b,
                                                                  const __grid_constant__ GemmArgs a) {
  using C = GemmCfg<PL>;
  constexpr int S = C::kStages;
  constexpr bool kAMN = USE == kWeight, kBMN = USE == kWeight || USE == kHidden;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  GemmBars* bars = reinterpret_cast<GemmBars*>(sm + (size_t)S * C::kStage);
  const CePlan& pl = a.pl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(bars->full + s, 1);
      ptx::mbar_init(bars->empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(bars->acc_full + b, 1);
      ptx::mbar_init(bars->acc_free + b, kEpiWarps);
    }
    ptx::mbar_init(&bars->done, 1);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&map_a);
    ptx::prefetch_tmap(&map_b);
  }
  if (warp == 2) {
    ptx::tmem_alloc(&bars->tmem, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem;
  griddep_wait();
  griddep_trigger();
  const int kept = *pl.kept;
  const Items<PL, USE> items(a, kept);
  const int n_items = items.count();

  if (warp == 0) {
    if (lane == 0) {   // ---------------------------------------------------- loads
      int it = 0;
      bool ok = true;
      // rows between the planes of each operand
      const int a_plane = pl.rows_pad, b_plane = USE == kWeight ? pl.rows_pad : pl.piece;
      for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x) {
        int m0, n0, b0, b1;
        items.get(item, m0, n0, b0, b1);
        // a bf16 head is read where the caller has it
        const int v0 = PL == 1 ? a.v0 : 0;
        for (int kb = b0; kb < b1; ++kb, ++it) {
          const int s = it % S;
          if (it >= S && !ptx::mbar_wait(bars->empty + s, ((it / S) & 1) ^ 1, kBudget, pl.status)) {
            ok = false;
            break;
          }
          uint8_t* st = sm + (size_t)s * C::kStage;
          ptx::mbar_arrive_expect_tx(bars->full + s, C::kStage);
#pragma unroll
          for (int p = 0; p < PL; ++p) {
            uint8_t* ta = st + p * C::kA;
            if (kAMN) {
#pragma unroll
              for (int i = 0; i < kBM / 64; ++i)
                tma_tile(ta + i * 8192, &map_a, bars->full + s, m0 + 64 * i, p * a_plane + kb * 64);
            } else {
              tma_tile(ta, &map_a, bars->full + s, kb * 64, p * a_plane + m0);
            }
            uint8_t* tb = st + PL * C::kA + p * C::kB;
            if (kBMN) {
              const int row = p * b_plane + (USE == kHidden ? v0 : 0) + kb * 64;
#pragma unroll
              for (int i = 0; i < C::kBN / 64; ++i) tma_tile(tb + i * 8192, &map_b, bars->full + s, n0 + 64 * i, row);
            } else {
              tma_tile(tb, &map_b, bars->full + s, kb * 64, p * b_plane + v0 + n0);
            }
          }
        }
      }
      // every load issued lands before the CTA can exit
      for (int j = max(0, it - S); j < it; ++j) ptx::mbar_wait(bars->full + j % S, (j / S) & 1, kBudget, nullptr);
    }
  } else if (warp == 1) {   // ---------------------------------------------- MMAs
    // The whole warp runs this, so that what it computes is uniform; one elected
    // lane issues each group of MMAs with the commits behind it.
    constexpr uint32_t id = ptx::idesc_bf16_f32(kBM, C::kBN) | (kAMN ? 1u << 15 : 0u) | (kBMN ? 1u << 16 : 0u);
    constexpr uint32_t ka = k_step<kAMN>(), kb_ = k_step<kBMN>();
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t p) {
      if (!__all_sync(0xffffffffu, ptx::mbar_try_wait(b, p))) {
        ok = ok && ptx::mbar_wait(b, p, kBudget, pl.status);
        ok = __all_sync(0xffffffffu, ok);
      }
      ptx::tc_fence_after();
      return ok;
    };
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t base = ptx::smem_u32(sm);
    int it = 0, seq = 0;
    for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x) {
      int m0, n0, b0, b1;
      items.get(item, m0, n0, b0, b1);
      for (int kb = b0; kb < b1 && ok; ++seq) {
        const int buf = seq & 1, use = seq >> 1;
        if (use >= 1 && !wait(bars->acc_free + buf, (use - 1) & 1)) break;
        const uint32_t d = tm + buf * C::kAccCols;
        const int end = min(kb + kSumBlocks, b1);
        uint32_t acc = 0;
        for (; kb < end; ++kb, ++it) {
          const int s = it % S;
          if (!wait(bars->full + s, (it / S) & 1)) break;
          const uint32_t da = desc_lo<kAMN>(base + s * C::kStage), db = desc_lo<kBMN>(base + s * C::kStage + PL * C::kA);
          if (elect()) {
            if constexpr (PL == 1) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mma(d, da + k * ka, db + k * kb_, id, acc | (k != 0));
            } else {
              // small products first: l h, h l, m m, m h, h m, then h h
              constexpr int qa[6] = {2, 0, 1, 1, 0, 0}, qb[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
              for (int q = 0; q < 6; ++q)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma(d + (q < 5 ? C::kBN : 0), da + (qa[q] * C::kA >> 4) + k * ka, db + (qb[q] * C::kB >> 4) + k * kb_,
                      id, acc | (k != 0) | (q > 0 && q < 5));
            }
            ptx::mma_commit(bars->empty + s);
            if (kb + 1 == end) ptx::mma_commit(bars->acc_full + buf);
          }
          __syncwarp();
          acc = 1;
        }
      }
    }
    if (elect()) ptx::mma_commit(&bars->done);
    __syncwarp();
    ptx::mbar_wait(&bars->done, 0, kBudget, nullptr);   // what was issued ends before the CTA does
  } else if (warp >= 4) {   // ---------------------------------------------- sums
    constexpr int NC = C::kNC;
    const int half = (warp - 4) >> 2, lane_row = 32 * (warp & 3) + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const int c_half = half * NC;
    int seq = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x) {
      int m0, n0, b0, b1;
      items.get(item, m0, n0, b0, b1);
      float acc[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j) acc[j] = 0.f;
      for (int kb = b0; kb < b1; kb += kSumBlocks, ++seq) {
        const int buf = seq & 1;
        if (!ptx::mbar_wait(bars->acc_full + buf, (seq >> 1) & 1, kBudget, pl.status)) ok = false;
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t at = tmem + lanes + buf * C::kAccCols + c_half;
#pragma unroll
        for (int j0 = 0; j0 < NC; j0 += 16) {
          float v[16];
          if constexpr (PL == 3) {
            ptx::tmem_ld16(at + C::kBN + j0, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[j0 + j] += v[j];
          }
          ptx::tmem_ld16(at + j0, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[j0 + j] += v[j];
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars->acc_free + buf);
      }
      if (!ok) break;
      const int row = m0 + lane_row;   // (a vocabulary row of the piece for kWeight)
      if constexpr (USE == kStats) {
        if (row < kept) {
          const int col = n0 + c_half;                       // within the piece
          const int left = a.cols - col;                     // columns that there are
          const int tgt = pl.target[row] - a.v0 - col;
          float m = -INFINITY, s = 0.f;
#pragma unroll
          for (int j0 = 0; j0 < NC; j0 += 32) {
            if (j0 >= left) break;
            float gm = -INFINITY;
#pragma unroll
            for (int j = j0; j < j0 + 32; ++j) {
              acc[j] *= a.scale2;
              if (j >= left) acc[j] = -INFINITY;
              if (j == tgt) pl.picked[row] = acc[j];
              gm = fmaxf(gm, acc[j]);
            }
            const float nm = fmaxf(m, gm), ref = nm == -INFINITY ? 0.f : nm;
            s *= ex2(m - ref);
            float part = 0.f;
#pragma unroll
            for (int j = j0; j < j0 + 32; ++j) part += ex2(acc[j] - ref);
            s += part;
            m = nm;
          }
          pl.part[(size_t)(a.part0 + 2 * (n0 / C::kBN) + half) * pl.rows_pad + row] = make_float2(m, s);
        }
      } else if constexpr (USE == kGrad) {
        const bool in = row < kept;
        const float2 l2 = in ? pl.lse2[row] : make_float2(0.f, 0.f);
        const float gain = in ? pl.gain[row] : 0.f;
        const int col = n0 + c_half, left = in ? a.cols - col : 0, tgt = in ? pl.target[row] - a.v0 - col : -1;
        __nv_bfloat16* out = pl.g + (size_t)row * pl.piece + col;
#pragma unroll
        for (int j0 = 0; j0 < NC; j0 += 8) {
          float g[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = j0 + j;
            float e = fmaf(acc[c], a.scale2, -l2.x);
            if (PL == 3) e = fmaf(acc[c], a.scale2_lo, e - l2.y);
            g[j] = c < left ? gain * (ex2(e) - (c == tgt ? 1.f : 0.f)) : 0.f;
          }
          put8<PL>(out + j0, (size_t)pl.rows_pad * pl.piece, g);
        }
      } else if constexpr (USE == kHidden) {
        float* out = pl.acc + ((size_t)items.split_of(item) * pl.rows_pad + row) * pl.dim_pad + n0 + c_half;
        const int left = pl.dim_pad - n0 - c_half;
#pragma unroll
        for (int j = 0; j < NC; j += 4) {
          if (j >= left) break;
          float4 v = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
          float4* p = reinterpret_cast<float4*>(out + j);
          if (!a.first) {
            const float4 o = *p;
            v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
          }
          *p = v;
        }
      } else {
        if (row < a.cols) {
          const size_t at = (size_t)(a.v0 + row) * pl.dim + n0 + c_half;
          const int left = pl.dim - n0 - c_half;   // a multiple of 8
#pragma unroll
          for (int j = 0; j < NC; j += 8) {
            if (j >= left) break;
            if (PL == 3) set8(static_cast<float*>(a.d_weight) + at + j, true, acc + j);
            else set8(static_cast<__nv_bfloat16*>(a.d_weight) + at + j, true, acc + j);
          }
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- ends
// A row's pairs merged: lse = ln2 (M + log2 S), and the loss from the difference of
// the exponents, which is exact where the target has the largest.
constexpr int kMergeWarps = 16;

__global__ void __launch_bounds__(32 * kMergeWarps) ce_merge_kernel(CePlan pl, int parts, float* loss, float* lse) {
  griddep_wait();
  griddep_trigger();
  __shared__ float2 sh[kMergeWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kept = *pl.kept;
  for (int r0 = blockIdx.x * 32; r0 < kept; r0 += gridDim.x * 32) {
    const int r = r0 + lane;
    float m = -INFINITY, s = 0.f;
    auto add = [&](float2 v) {
      const float nm = fmaxf(m, v.x), ref = nm == -INFINITY ? 0.f : nm;
      s = s * ex2(m - ref) + v.y * ex2(v.x - ref);
      m = nm;
    };
    if (r < kept) {
      int p = warp;
      for (; p + 3 * kMergeWarps < parts; p += 4 * kMergeWarps) {
        float2 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = pl.part[(size_t)(p + u * kMergeWarps) * pl.rows_pad + r];
#pragma unroll
        for (int u = 0; u < 4; ++u) add(v[u]);
      }
      for (; p < parts; p += kMergeWarps) add(pl.part[(size_t)p * pl.rows_pad + r]);
    }
    __syncthreads();
    sh[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (warp == 0 && r < kept) {
      m = -INFINITY;
      s = 0.f;
      for (int w = 0; w < kMergeWarps; ++w) add(sh[w][lane]);
      const float l2 = log2f(s);
      const int to = pl.row_of[r];
      lse[to] = kLn2 * (m + l2);
      loss[to] = kLn2 * ((m - pl.picked[r]) + l2);
    }
  }
}

// The shares of the hidden states' gradient added in order, to the caller's rows.
template <typename T>
__global__ void __launch_bounds__(256) ce_finish_hidden_kernel(CePlan pl, T* d_hidden, int64_t stride) {
  griddep_wait();
  griddep_trigger();
  const int kept = *pl.kept, groups = pl.dim / 8;
  const bool vec = rows_vec(d_hidden, stride);
  const size_t share = (size_t)pl.rows_pad * pl.dim_pad;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < (long long)kept * groups; i += gridDim.x * 256LL) {
    const int r = (int)(i / groups), c = (int)(i - (long long)r * groups) * 8;
    const float* src = pl.acc + (size_t)r * pl.dim_pad + c;
    float sum[8];
    get8(src, true, sum);
    for (int s = 1; s < pl.splits; ++s) {
      float v[8];
      get8(src + s * share, true, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += v[j];
    }
    set8(d_hidden + pl.row_of[r] * stride + c, vec, sum);
  }
}

// ---------------------------------------------------------------- host side
template <int PL>
cudaError_t prepare() {
  for (auto kernel : {ce_gemm_kernel<PL, kStats>, ce_gemm_kernel<PL, kGrad>, ce_gemm_kernel<PL, kHidden>, ce_gemm_kernel<PL, kWeight>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)GemmCfg<PL>::kBytes);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int PL, int USE>
cudaError_t gemm(const GemmArgs& a, const CUtensorMap& ma, const CUtensorMap& mb, int sms, int* launches, cudaStream_t s) {
  ++*launches;
  return launch_pdl(ce_gemm_kernel<PL, USE>, dim3(sms), dim3(kGemmThreads), GemmCfg<PL>::kBytes, s, ma, mb, a);
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

template <typename T, int PL>
cudaError_t forward(const CePlan& pl, const CeTensors& t, int sms, int* launches, cudaStream_t s) {
  using C = GemmCfg<PL>;
  const int per = gather_rows(pl.rows);
  cudaError_t e = launch_pdl(ce_gather_kernel<T, PL, false>, dim3((pl.rows + per - 1) / per), dim3(kGatherThreads), 0, s, pl, t, per);
  ++*launches;
  if (e != cudaSuccess) return e;
  CUtensorMap mh, mw;
  bool ok = encode_activation_map(&mh, pl.h, pl.dim_pad, PL * pl.rows_pad, pl.dim_pad, kBM);
  ok = ok && (PL == 1 ? encode_activation_map(&mw, t.weight, pl.dim, pl.vocab, pl.dim, C::kBN)
                      : encode_activation_map(&mw, pl.w, pl.dim_pad, PL * pl.piece, pl.dim_pad, C::kBN));
  if (!ok) return cudaErrorInvalidValue;
  GemmArgs a{};
  a.pl = pl;
  const Scale sc = scale_of(t.temperature);
  a.scale2 = sc.hi;
  a.scale2_lo = sc.lo;
  for (int v0 = 0; v0 < pl.vocab; v0 += pl.piece) {
    a.v0 = v0;
    a.cols = std::min(pl.piece, pl.vocab - v0);
    if (PL == 3) {
      e = launch_pdl(ce_split_weight_kernel, dim3(sms * 8), dim3(256), 0, s, pl, static_cast<const float*>(t.weight), v0);
      ++*launches;
      if (e != cudaSuccess) return e;
    }
    e = gemm<PL, kStats>(a, mh, mw, sms, launches, s);
    if (e != cudaSuccess) return e;
    a.part0 += 2 * ((a.cols + C::kBN - 1) / C::kBN);
  }
  ++*launches;
  return launch_pdl(ce_merge_kernel, dim3((pl.rows + 31) / 32), dim3(32 * kMergeWarps), 0, s, pl, a.part0, t.loss, t.lse);
}

template <typename T, int PL>
cudaError_t backward(const CePlan& pl, const CeTensors& t, int sms, int* launches, cudaStream_t s) {
  using C = GemmCfg<PL>;
  const int per = gather_rows(pl.rows);
  cudaError_t e = launch_pdl(ce_gather_kernel<T, PL, true>, dim3((pl.rows + per - 1) / per), dim3(kGatherThreads), 0, s, pl, t, per);
  ++*launches;
  if (e != cudaSuccess) return e;
  // operands with the product's K along their rows (boxes of 64 x rows of the tile) or across them (64 x 64)
  CUtensorMap h_k, h_mn, w_k, w_mn, g_k, g_mn;
  const void* w = PL == 1 ? t.weight : pl.w;
  const int w_dim = PL == 1 ? pl.dim : pl.dim_pad, w_rows = PL == 1 ? pl.vocab : PL * pl.piece;
  if (!encode_activation_map(&h_k, pl.h, pl.dim_pad, PL * pl.rows_pad, pl.dim_pad, kBM) ||
      !encode_activation_map(&h_mn, pl.h, pl.dim_pad, PL * pl.rows_pad, pl.dim_pad, 64) ||
      !encode_activation_map(&w_k, w, w_dim, w_rows, w_dim, C::kBN) ||
      !encode_activation_map(&w_mn, w, w_dim, w_rows, w_dim, 64) ||
      !encode_activation_map(&g_k, pl.g, pl.piece, PL * pl.rows_pad, pl.piece, kBM) ||
      !encode_activation_map(&g_mn, pl.g, pl.piece, PL * pl.rows_pad, pl.piece, 64))
    return cudaErrorInvalidValue;
  GemmArgs a{};
  a.pl = pl;
  const Scale sc = scale_of(t.temperature);
  a.scale2 = sc.hi;
  a.scale2_lo = sc.lo;
  a.d_weight = t.d_weight;
  for (int v0 = 0; v0 < pl.vocab; v0 += pl.piece) {
    a.v0 = v0;
    a.cols = std::min(pl.piece, pl.vocab - v0);
    a.first = v0 == 0;
    if (PL == 3) {
      e = launch_pdl(ce_split_weight_kernel, dim3(sms * 8), dim3(256), 0, s, pl, static_cast<const float*>(t.weight), v0);
      ++*launches;
      if (e != cudaSuccess) return e;
    }
    if ((e = gemm<PL, kGrad>(a, h_k, w_k, sms, launches, s)) != cudaSuccess) return e;
    if (t.d_hidden && (e = gemm<PL, kHidden>(a, g_k, w_mn, sms, launches, s)) != cudaSuccess) return e;
    if (t.d_weight && (e = gemm<PL, kWeight>(a, g_mn, h_mn, sms, launches, s)) != cudaSuccess) return e;
  }
  if (!t.d_hidden) return cudaSuccess;
  ++*launches;
  const long long groups = (long long)pl.rows * (pl.dim / 8);
  return launch_pdl(ce_finish_hidden_kernel<T>, dim3((unsigned)std::min<long long>((groups + 255) / 256, sms * 8)), dim3(256), 0,
                    s, pl, static_cast<T*>(t.d_hidden), t.d_row_stride);
}

}  // namespace

CePlan ce_plan(void* ws, int rows, int dim, int vocab, bool f32, bool backward, bool want_hidden, int sms) {
  CePlan pl{};
  pl.rows = rows;
  pl.dim = dim;
  pl.vocab = vocab;
  pl.planes = f32 ? 3 : 1;
  pl.rows_pad = (rows + kBM - 1) / kBM * kBM;
  pl.dim_pad = (dim + 63) / 64 * 64;
  const int bn = f32 ? GemmCfg<3>::kBN : GemmCfg<1>::kBN;
  // pieces of equal size, as few as the limit allows
  const size_t column = 2 * (size_t)pl.planes * (backward ? std::max(pl.rows_pad, f32 ? pl.dim_pad : 0) : pl.dim_pad);
  const long long limit = std::max<long long>(256, (long long)(kPieceBytes / column) / 256 * 256);
  const long long all = ((long long)vocab + 255) / 256 * 256;
  if (!backward && !f32) {
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
  if (f32) pl.w = reinterpret_cast<__nv_bfloat16*>(take(6 * (size_t)pl.piece * pl.dim_pad));
  pl.splits = 1;
  if (!backward) {
    const size_t pieces = (size_t)((vocab + pl.piece - 1) / pl.piece);
    pl.part = reinterpret_cast<float2*>(take(sizeof(float2) * 2 * pieces * ((pl.piece + bn - 1) / bn) * R));
    pl.picked = reinterpret_cast<float*>(take(4 * R));
  } else {
    pl.lse2 = reinterpret_cast<float2*>(take(8 * R));
    pl.gain = reinterpret_cast<float*>(take(4 * R));
    pl.g = reinterpret_cast<__nv_bfloat16*>(take(2 * pl.planes * R * pl.piece));
    if (want_hidden) {
      // shares of a piece's columns: as many as fill the SMs evenly, against the fp32 sums' traffic
      const double tiles = (double)(R / kBM) * ((dim + bn - 1) / bn), blocks = pl.piece / 64;
      double best = 1e300;
      for (int n = 1; n <= 64 && n <= blocks; ++n) {
        const double items = std::ceil(tiles * n / sms) * (std::ceil(blocks / n) * (f32 ? 1600 : 550) + 4000);
        const double sums = n * tiles * kBM * bn * 8.0 / 3500.0;   // bytes over bytes a cycle
        if (items + sums < best * 0.98) {
          best = items + sums;
          pl.splits = n;
        }
      }
      pl.acc = reinterpret_cast<float*>(take(4 * (size_t)pl.splits * R * pl.dim_pad));
    }
  }
  pl.bytes = off;
  return pl;
}

cudaError_t ce_prepare_f32() { return prepare<3>(); }
cudaError_t ce_prepare_bf16() { return prepare<1>(); }

cudaError_t ce_forward(const CePlan& pl, const CeTensors& t, int sms, int* launches, cudaStream_t s) {
  *launches = 0;
  return pl.planes == 3 ? forward<float, 3>(pl, t, sms, launches, s) : forward<__nv_bfloat16, 1>(pl, t, sms, launches, s);
}

cudaError_t ce_backward(const CePlan& pl, const CeTensors& t, int sms, int* launches, cudaStream_t s) {
  *launches = 0;
  return pl.planes == 3 ? backward<float, 3>(pl, t, sms, launches, s) : backward<__nv_bfloat16, 1>(pl, t, sms, launches, s);
}

}  // namespace dflash
