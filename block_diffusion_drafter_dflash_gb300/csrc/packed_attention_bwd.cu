// Gradients of the packed training attention (the forward is
// packed_attention.cu; paper section 4.2).  For a query row r (block n, position i,
// query head h) and the keys j it sees (context keys below the block's anchor,
// then the block's own), with P = exp(s - lse):
//
//   s = q.k / sqrt(hd)     D = sum_d d_out out     dp = d_out.v
//   ds = P (dp - D)        dq = sum_j ds k / sqrt(hd)
//   dk = sum_r ds q / sqrt(hd)      dv = sum_r P d_out
//
// A context key collects from every block anchored behind it and from the
// G = nq / nkv query heads that share it; a block key from its own block.
//
// Sorted by anchor, the blocks a key tile is seen by are the last ones, and the
// keys a row tile sees are the first ones: no mask is stored and only tiles that
// a boundary crosses compare positions.  Row tiles hold whole blocks, so a
// block's own keys are the same places of the row tile's own key tile.
//
// One launch does the work, every CTA one of three kinds of item:
//   context keys  (q head, 128 keys, split): for each row tile that sees them
//                 S' = K Q', dP' = V dO'  (keys on the tensor-memory lanes),
//                 dV += P' dO, dK += dS' Q, with P' and dS' written back to tensor
//                 memory as the A operand; its share goes to memory as fp32 and a
//                 last kernel adds the shares of heads and splits in order;
//   rows          (q head, 128 rows): for each key tile S = Q K', dP = dO V',
//                 dQ += dS K;
//   own keys      (kv head, row tile): as context keys, over the G heads.
// S and dP are thus computed twice (7 products instead of 5), and nothing is
// accumulated with atomics: the results do not change from run to run.
//
// In a CTA one thread loads tiles by TMA, one issues the MMAs, and eight warps
// turn S and dP into P and dS.  The MMA thread alternates so that the tensor
// cores work on the other product while the eight warps work on one:
//   keys:  dV(i) S(i+1) | dK(i) dP(i+1)      rows:  S(i+1) dP(i+1) dQ(i)
// Each operand tile is staged once and read in both directions: K-major for S and
// dP, MN-major as the B operand of the gradients.
//
// Operands, P and dS enter the products as fp16, which has three more bits than
// bf16, scaled by powers of two so that its range holds them: q, k, v and d_out
// each by the power that brings its largest value to 2^14 .. 2^15, P (at most 1) by
// 2^14, and ds by what the largest norms of d_out's and v's rows allow it
// (|dp| <= |d_out_r| |v_j|).  The scales are folded into factors that are there
// anyway, and powers of two are exact.  bf16 tensors take one plane: the operands
// are then exact but for d_out, and d_out, P and ds are rounded by 2^-12 of
// themselves, an eighth of the rounding of the bf16 gradients.  fp32 tensors
// take each operand, P and ds included, as a hi + lo pair (22 bits) and each
// product as three MMAs (hi hi, hi lo, lo hi).  Every sum and the softmax are fp32.
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "gemm.cuh"
#include "packed_attention_bwd.cuh"
#include "ptx.cuh"

namespace dflash {
namespace {

constexpr int kRows = 128;           // rows of a row tile, keys of a key tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr long long kBudget = 400000000LL;
constexpr int kOpExp = 14;           // an operand's largest value lies in [2^14, 2^15)
constexpr int kPExp = 14;            // P is held times 2^14
constexpr int kRangeValues = 6;      // largest |q|, |k|, |v|, |d_out|, and largest norm of a row of v, d_out
constexpr int kRangeThreads = 512;

// Exponents e of the scales 2^e of q, k, v and d_out, and of dp (and D):
// ds is held as P 2^14 (dp - D) 2^dp.
struct Scales {
  int q, k, v, o, dp;
};
__device__ __forceinline__ float pow2(int e) { return ldexpf(1.f, e); }
// The exponent that brings m into [2^14, 2^15), within what a float holds.
__device__ __forceinline__ int scale_exp(float m) {
  if (!(m > 0.f) || isinf(m)) return 0;
  return max(-120, min(120, kOpExp - ilogbf(m)));
}
__device__ __forceinline__ Scales scales_of(const float* m) {
  Scales s;
  s.q = scale_exp(m[0]);
  s.k = scale_exp(m[1]);
  s.v = scale_exp(m[2]);
  s.o = scale_exp(m[3]);
  // |dp - D| <= 2 |d_out| |v| by the rows' norms
  auto norm_exp = [](float n) { return n > 0.f && !isinf(n) ? ilogbf(n) + 1 : 0; };
  s.dp = -(norm_exp(m[4]) + norm_exp(m[5]) + 1);
  return s;
}
__device__ __forceinline__ Scales load_scales(const int32_t* p) { return Scales{p[0], p[1], p[2], p[3], p[4]}; }

// ---------------------------------------------------------------- loads
// E (2 or 4) consecutive values, in one load where their address allows it.
template <int E>
__device__ __forceinline__ void load_values(const float* p, float* v) {
  if (reinterpret_cast<uintptr_t>(p) % (4 * E) == 0) {
    if constexpr (E == 4) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(p));
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const float2 x = __ldcs(reinterpret_cast<const float2*>(p));
      v[0] = x.x, v[1] = x.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = p[e];
  }
}
template <int E>
__device__ __forceinline__ void load_values(const __nv_bfloat16* p, float* v) {
  if (reinterpret_cast<uintptr_t>(p) % (2 * E) == 0) {
    uint32_t w[E / 2];
    if constexpr (E == 4) {
      const uint2 x = __ldcs(reinterpret_cast<const uint2*>(p));
      w[0] = x.x, w[1] = x.y;
    } else {
      w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    }
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = __bfloat162float(p[e]);
  }
}

// ---------------------------------------------------------------- anchors in order, ranges of the operands
// Place of block n: how many blocks have a smaller anchor, or the same and a
// smaller number.  Anchors outside [0, S] are clamped and flagged.
__device__ void rank_blocks(const PackedBwdPlan& pl, const int32_t* anchors, int cta) {
  __shared__ int32_t tile[1024];
  const int n = cta * kRangeThreads + threadIdx.x;
  const int own = n < pl.N ? min(max(anchors[n], 0), pl.S) : 0;
  int rank = 0, bad = 0;
  for (int base = 0; base < pl.N; base += 1024) {
    const int cnt = min(1024, pl.N - base);
    __syncthreads();
    for (int i = threadIdx.x; i < cnt; i += kRangeThreads) {
      const int a = anchors[base + i];
      bad |= a < 0 || a > pl.S;
      tile[i] = min(max(a, 0), pl.S);
    }
    __syncthreads();
    for (int i = 0; i < cnt; ++i) rank += tile[i] < own || (tile[i] == own && base + i < n);
  }
  bad = __syncthreads_or(bad);
  if (cta == 0 && threadIdx.x == 0) *pl.status = bad ? DFLASH_ERR_INVALID_ARG : 0;
  if (n < pl.N) {
    pl.order[rank] = n;
    pl.sorted[rank] = own;
  }
}

// Largest value (and, where NORM, largest norm of a row) of `rows` rows of
// HD values; a warp takes four rows at a time.
template <typename T, int HD, bool NORM>
__device__ __forceinline__ void range_rows(const T* x, long long rows, int part, int parts, float& mx, float& nm) {
  constexpr int E = HD / 32, U = 4;
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)parts * (kRangeThreads / 32);
  for (long long r0 = ((long long)part * (kRangeThreads / 32) + (threadIdx.x >> 5)) * U; r0 < rows; r0 += warps * U) {
    float v[U][E] = {};
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r0 + u < rows) load_values<E>(x + (size_t)(r0 + u) * HD + E * lane, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        mx = fmaxf(mx, fabsf(v[u][e]));
        if (NORM) sq = fmaf(v[u][e], v[u][e], sq);
      }
      if (NORM) {
#pragma unroll
        for (int o = 16; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        if (sq > 1.0e-30f && sq < 1.0e36f) {
          nm = fmaxf(nm, sqrtf(sq));
        } else {   // zeros, or squares outside fp32's range: over the row's largest value
          float top = 0.f, s2 = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(v[u][e]));
          for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (top > 0.f) {
#pragma unroll
            for (int e = 0; e < E; ++e) s2 = fmaf(v[u][e] / top, v[u][e] / top, s2);
            for (int o = 16; o; o >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
            nm = fmaxf(nm, top * sqrtf(s2));
          }
        }
      }
    }
  }
}

// The first CTAs put the blocks in order, the others look for the operands'
// ranges (one row of maxima each, merged by the next kernel).
template <typename T, int HD>
__global__ void __launch_bounds__(kRangeThreads) range_kernel(PackedBwdPlan pl, PackedBwdTensors t) {
  griddep_wait();
  griddep_trigger();
  const int rank_ctas = (pl.N + kRangeThreads - 1) / kRangeThreads;
  if ((int)blockIdx.x < rank_ctas) {
    rank_blocks(pl, t.anchors, blockIdx.x);
    return;
  }
  const int part = blockIdx.x - rank_ctas, parts = pl.parts;
  float m[kRangeValues] = {};
  float none = 0.f;
  const long long qr = (long long)pl.N * pl.block * pl.nq, br = (long long)pl.N * pl.block * pl.nkv,
                  cr = (long long)pl.S * pl.nkv;
  range_rows<T, HD, false>(static_cast<const T*>(t.q), qr, part, parts, m[0], none);
  range_rows<float, HD, true>(t.d_out, qr, part, parts, m[3], m[5]);
  range_rows<T, HD, false>(static_cast<const T*>(t.k_blk), br, part, parts, m[1], none);
  range_rows<T, HD, true>(static_cast<const T*>(t.v_blk), br, part, parts, m[2], m[4]);
  range_rows<T, HD, false>(static_cast<const T*>(t.k_ctx), cr, part, parts, m[1], none);
  range_rows<T, HD, true>(static_cast<const T*>(t.v_ctx), cr, part, parts, m[2], m[4]);
  __shared__ float sh[kRangeThreads / 32][kRangeValues];
#pragma unroll
  for (int i = 0; i < kRangeValues; ++i) {
#pragma unroll
    for (int o = 16; o; o >>= 1) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5][i] = m[i];
  }
  __syncthreads();
  if (threadIdx.x < kRangeValues) {
    float x = 0.f;
    for (int w = 0; w < kRangeThreads / 32; ++w) x = fmaxf(x, sh[w][threadIdx.x]);
    pl.part[part * kRangeValues + threadIdx.x] = x;
  }
}

// ---------------------------------------------------------------- operand layout
// E = hd / 32 values of a lane times `scale`, as one or two fp16 planes `plane`
// apart; v becomes what the planes hold.
template <int E>
__device__ __forceinline__ void put_planes(__half* dst, size_t plane, int planes, float scale, float* v) {
  __half2 h[E / 2], l[E / 2];
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float x = v[e] * scale, y = v[e + 1] * scale;
    h[e / 2] = __floats2half2_rn(x, y);
    float2 f = __half22float2(h[e / 2]);
    l[e / 2] = __floats2half2_rn(x - f.x, y - f.y);
    v[e] = f.x;
    v[e + 1] = f.y;
    if (planes == 2) {
      f = __half22float2(l[e / 2]);
      v[e] += f.x;
      v[e + 1] += f.y;
    }
  }
  auto put = [&](__half* d, const __half2* x) {
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(d) = *reinterpret_cast<const uint2*>(x);
    else
      *reinterpret_cast<uint32_t*>(d) = *reinterpret_cast<const uint32_t*>(x);
  };
  put(dst, h);
  if (planes == 2) put(dst + plane, l);
}

// One warp per row: query rows (with D and lse), then the blocks' own keys and
// values, then the context's.  Bound by HBM: q, out and d_out are read once.
template <typename T, int HD>
__global__ void __launch_bounds__(256) pack_bwd_kernel(PackedBwdPlan pl, PackedBwdTensors t) {
  griddep_wait();
  griddep_trigger();
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31, g = pl.block, rows = pl.T * kRows, ctx = pl.KT * kRows;
  const long long n_q = (long long)rows * pl.nq, n_b = (long long)rows * pl.nkv, n_c = (long long)ctx * pl.nkv;
  const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
  // the CTAs' maxima become the scales
  __shared__ float s_max[kRangeValues];
  __shared__ Scales s_sc;
  if (threadIdx.x < 32 * kRangeValues) {
    const int i = threadIdx.x >> 5;
    float x = 0.f;
    for (int p = lane; p < pl.parts; p += 32) x = fmaxf(x, pl.part[p * kRangeValues + i]);
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    if (lane == 0) s_max[i] = x;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    s_sc = scales_of(s_max);
    if (blockIdx.x == 0) {
      pl.scale[0] = s_sc.q;
      pl.scale[1] = s_sc.k;
      pl.scale[2] = s_sc.v;
      pl.scale[3] = s_sc.o;
      pl.scale[4] = s_sc.dp;
    }
  }
  __syncthreads();
  const float f_q = pow2(s_sc.q), f_k = pow2(s_sc.k), f_v = pow2(s_sc.v), f_o = pow2(s_sc.o);
  const int e_d = s_sc.dp - s_sc.o;   // D is summed over the scaled d_out
  // block and position of a row; -1: padding
  auto place = [&](int r, int& n, int& i) {
    const int k = r % kRows, b = k / g, at = (r / kRows) * pl.per + b;
    n = b < pl.per && at < pl.N ? pl.order[at] : -1;
    i = k - b * g;
    return at;
  };
  for (long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < n_q + n_b + n_c; w += warps) {
    float a[E] = {}, b[E] = {}, c[E] = {};
    if (w < n_q) {
      const int h = (int)(w % pl.nq), r = (int)(w / pl.nq);
      int n, i;
      const int at = place(r, n, i);
      float d = 0.f, l = INFINITY;
      if (n >= 0) {
        const size_t row = ((size_t)n * g + i) * pl.nq + h, o = row * HD + E * lane;
        load_values<E>(static_cast<const T*>(t.q) + o, a);
        load_values<E>(t.d_out + o, b);
        load_values<E>(t.out + o, c);
        l = fmaf(t.lse[row], kLog2e, -(float)kPExp);
      }
      const size_t dst = ((size_t)h * pl.planes * rows + r) * HD + E * lane, plane = (size_t)rows * HD;
      put_planes<E>(pl.q + dst, plane, pl.planes, f_q, a);
      put_planes<E>(pl.d_o + dst, plane, pl.planes, f_o, b);
      // D from d_out as the products see it: its rounding then cancels in dp - D as exactly as d_out itself would
#pragma unroll
      for (int e = 0; e < E; ++e) d = fmaf(b[e], c[e], d);
      for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      if (lane == 0) {
        pl.lse2[(size_t)h * rows + r] = l;
        pl.delta[(size_t)h * rows + r] = ldexpf(d, e_d);
        if (h == 0) pl.row_anchor[r] = n >= 0 ? pl.sorted[at] : 0;
      }
    } else if (w < n_q + n_b) {
      const long long u = w - n_q;
      const int h = (int)(u % pl.nkv), r = (int)(u / pl.nkv);
      int n, i;
      place(r, n, i);
      if (n >= 0) {
        const size_t o = (((size_t)n * g + i) * pl.nkv + h) * HD + E * lane;
        load_values<E>(static_cast<const T*>(t.k_blk) + o, a);
        load_values<E>(static_cast<const T*>(t.v_blk) + o, b);
      }
      const size_t dst = ((size_t)h * pl.planes * rows + r) * HD + E * lane, plane = (size_t)rows * HD;
      put_planes<E>(pl.kb + dst, plane, pl.planes, f_k, a);
      put_planes<E>(pl.vb + dst, plane, pl.planes, f_v, b);
    } else {
      const long long u = w - n_q - n_b;
      const int h = (int)(u % pl.nkv), r = (int)(u / pl.nkv);
      if (r < pl.S) {
        const size_t o = ((size_t)r * pl.nkv + h) * HD + E * lane;
        load_values<E>(static_cast<const T*>(t.k_ctx) + o, a);
        load_values<E>(static_cast<const T*>(t.v_ctx) + o, b);
      }
      const size_t dst = ((size_t)h * pl.planes * ctx + r) * HD + E * lane, plane = (size_t)ctx * HD;
      put_planes<E>(pl.kc + dst, plane, pl.planes, f_k, a);
      put_planes<E>(pl.vc + dst, plane, pl.planes, f_v, b);
    }
  }
}

// ---------------------------------------------------------------- tensor-core pieces
// Instruction descriptor, kind::f16: fp16 A and B, fp32 D, M x N (formats of
// A and B zero; both K-major).
constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] B[smem], fp16 in, fp32 out: A's rows on the lanes, two
// consecutive K values to a 32-bit column.
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A tile of rows of 64 fp16 (128-byte swizzle) as an MN-major operand: the 64
// values of a row run along N, the rows along K.  lbo: bytes to the tile of the
// next 64 values; 8 rows are 1024 bytes.
__device__ __forceinline__ uint64_t smem_desc_mn(const void* tile, int lbo) {
  const uint64_t addr = ptx::smem_u32(tile);
  return ((addr >> 4) & 0x3FFFull) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
constexpr uint32_t kBMajorMN = 1u << 16;   // instruction descriptor: B is MN-major

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   ptx::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 values as 16 columns of fp16 pairs from column `at` on and, with two
// planes, their rounding residuals in the next 16: the 32 columns that the
// values were read from.
template <int PL>
__device__ __forceinline__ void put_pairs(uint32_t at, const float* v) {
  uint32_t h[16], l[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    __half2 b = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
    h[j] = *reinterpret_cast<uint32_t*>(&b);
    if (PL == 2) {
      const float2 f = __half22float2(b);
      __half2 r = __floats2half2_rn(v[2 * j] - f.x, v[2 * j + 1] - f.y);
      l[j] = *reinterpret_cast<uint32_t*>(&r);
    }
  }
  tmem_st16(at, h);
  if (PL == 2) tmem_st16(at + 16, l);
}

// ---------------------------------------------------------------- the gradient kernel
// Warps 0..7 softmax (warp w: lanes 32 (w % 4), columns of half w / 4), warp 8
// loads, warp 9 issues the MMAs.
constexpr int kSoftWarps = 8;
constexpr int kGradThreads = 32 * (kSoftWarps + 2);

template <int HD, int PL>
struct GradCfg {
  static constexpr int kSub = HD / 64;
  // N of a streamed tile and the stages that fit beside the resident operands
  static constexpr int kN = PL == 2 && HD == 128 ? 64 : 128;
  static constexpr int kStages = PL == 2 && HD == 128 ? 1 : 2;
  static constexpr int kResTile = kRows * 128;             // 128 rows x 64 values
  static constexpr int kRes = PL * kSub * kResTile;        // one resident operand
  static constexpr int kStrTile = kN * 128;
  static constexpr int kStr = PL * kSub * kStrTile;        // one streamed operand
  static constexpr int kStat = 3 * kN * 4;                 // lse2, delta, anchors of a stage's rows
  static constexpr int kOffStr = 2 * kRes;
  static constexpr int kOffStat = kOffStr + kStages * 2 * kStr;
  static constexpr int kOffBars = kOffStat + kStages * kStat;
  static constexpr int kUsed = 1024 + kOffBars + 256;
  // more than half of an SM's shared memory: the CTA takes all of tensor memory
  static constexpr int kBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static constexpr int kHalf = kN / 2;                     // columns of S of one softmax warp
  static constexpr uint32_t kTmem = 512;
};

struct GradBars {
  uint64_t res_full, full[2], freed[2], s_full, dp_full, p_ready, ds_ready, done;
  uint32_t tmem;
};

struct GradMaps {
  CUtensorMap q, d_o, kc, vc, kb, vb;   // boxes of 64 values x 128 rows
  CUtensorMap qs, d_os, kcs, vcs, kbs, vbs;   // x kN rows (streamed)
};

template <typename T>
__device__ __forceinline__ void store32(T* dst, const float* v) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(dst + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
  } else {
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 b = __floats2bfloat162_rn(v[j + 2 * i], v[j + 2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(dst + j) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// S (+)= A B' over hd: A 128 resident rows, B kN streamed rows, both K-major.
template <int HD, int PL>
__device__ __forceinline__ void mma_scores(uint32_t d, const uint8_t* res, const uint8_t* str) {
  using C = GradCfg<HD, PL>;
  constexpr uint32_t id = idesc_f16(kRows, C::kN);
  uint32_t acc = 0;
#pragma unroll
  for (int pr = 0; pr < (PL == 2 ? 3 : 1); ++pr) {   // hi hi, hi lo, lo hi
    const int pa = pr == 2, pb = pr == 1;
#pragma unroll
    for (int s = 0; s < C::kSub; ++s)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ptx::mma_bf16(d, ptx::smem_desc_sw128(res + (pa * C::kSub + s) * C::kResTile) + 2 * k,
                      ptx::smem_desc_sw128(str + (pb * C::kSub + s) * C::kStrTile) + 2 * k, id, acc);
        acc = 1;
      }
  }
}
// G (+)= A B: A the P or dS of 128 lanes in tensor memory (columns of `a` as
// put_pairs left them), B kN streamed rows read along their values.
template <int HD, int PL>
__device__ __forceinline__ void mma_gradient(uint32_t d, uint32_t a, const uint8_t* str, uint32_t accumulate) {
  using C = GradCfg<HD, PL>;
  constexpr uint32_t id = idesc_f16(kRows, HD) | kBMajorMN;
  uint32_t acc = accumulate;
#pragma unroll
  for (int pr = 0; pr < (PL == 2 ? 3 : 1); ++pr) {
    const int pa = pr == 2, pb = pr == 1;
#pragma unroll
    for (int k = 0; k < C::kN / 16; ++k) {
      mma_tmem_a(d, a + (k >> 1) * 32 + pa * 16 + (k & 1) * 8,
                 smem_desc_mn(str + pb * C::kSub * C::kStrTile + k * 2048, C::kStrTile), id, acc);
      acc = 1;
    }
  }
}

template <typename T, int HD, int PL>
__global__ void __launch_bounds__(kGradThreads, 1) packed_grad_kernel(const __grid_constant__ PackedBwdPlan pl,
                                                                      const __grid_constant__ PackedBwdTensors t,
                                                                      const __grid_constant__ GradMaps maps) {
  using C = GradCfg<HD, PL>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  GradBars* bars = reinterpret_cast<GradBars*>(sm + C::kOffBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    ptx::mbar_init(&bars->res_full, 1);
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&bars->full[s], 1);
      ptx::mbar_init(&bars->freed[s], 1);
    }
    ptx::mbar_init(&bars->s_full, 1);
    ptx::mbar_init(&bars->dp_full, 1);
    ptx::mbar_init(&bars->p_ready, kSoftWarps);
    ptx::mbar_init(&bars->ds_ready, kSoftWarps);
    ptx::mbar_init(&bars->done, 1);
    ptx::fence_mbar_init();
  }
  if (warp == 0) {
    ptx::tmem_alloc(&bars->tmem, C::kTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem;
  griddep_wait();
  griddep_trigger();

  // ---- this CTA's item
  const int G = pl.nq / pl.nkv, rows = pl.T * kRows, ctx = pl.KT * kRows;
  constexpr int kPer = kRows / C::kN;        // streamed pieces of a 128-row tile
  const int n_ctx = pl.KT * pl.nq * pl.splits, n_rows = pl.T * pl.nq;
  int kind, h, tile, split = 0;              // kind 0: context keys, 1: rows, 2: own keys (h: kv head)
  {
    int b = blockIdx.x;
    if (b < n_ctx) {                         // the first keys are seen by most: longest items first
      kind = 0;
      tile = b / (pl.nq * pl.splits);
      b -= tile * pl.nq * pl.splits;
      h = b / pl.splits;
      split = b - h * pl.splits;
    } else if (b < n_ctx + n_rows) {
      kind = 1;
      b -= n_ctx;
      tile = pl.T - 1 - b / pl.nq;
      h = b % pl.nq;
    } else {
      kind = 2;
      b -= n_ctx + n_rows;
      tile = b / pl.nkv;
      h = b % pl.nkv;
    }
  }
  const int kvh = kind == 2 ? h : h / G;
  // streamed pieces [u0, u1): kind 0: of the rows; 1: of the context, then of
  // the own keys; 2: of the row tile, for each head in turn
  int u0 = 0, u1 = 0, ctx_pieces = 0;
  if (kind == 0) {
    // first row tile whose last block is anchored behind this tile's first key
    int lo = 0, hi = pl.T;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (pl.sorted[min((mid + 1) * pl.per, pl.N) - 1] > tile * kRows) hi = mid; else lo = mid + 1;
    }
    const int n = (pl.T - lo) * kPer;
    u0 = lo * kPer + (int)((long long)n * split / pl.splits);
    u1 = lo * kPer + (int)((long long)n * (split + 1) / pl.splits);
  } else if (kind == 1) {
    const int last = pl.sorted[min((tile + 1) * pl.per, pl.N) - 1];   // its largest anchor
    ctx_pieces = (last + C::kN - 1) / C::kN;
    u1 = ctx_pieces + kPer;
  } else {
    u1 = G * kPer;
  }
  const int n = u1 - u0;
  // streamed rows of piece u: (slab, first row) for kind 0 and 2 in [nq][planes][rows]
  auto piece_head = [&](int u) { return kind == 0 ? h : h * G + u / kPer; };
  auto piece_row = [&](int u) { return kind == 0 ? u * C::kN : tile * kRows + (u % kPer) * C::kN; };

  uint8_t* str = sm + C::kOffStr;
  auto stage = [&](int i) { return str + (i % C::kStages) * 2 * C::kStr; };
  auto stats = [&](int i) { return reinterpret_cast<float*>(sm + C::kOffStat + (i % C::kStages) * C::kStat); };
  auto par = [&](int i) { return static_cast<uint32_t>(i / C::kStages) & 1u; };
  const uint32_t tA = tmem, tB = tmem + 256;
  // kind 0, 2: S in columns [0, kN), dP at 128, dV at 256, dK at 256 + HD.
  // kind 1: S in two buffers at 0 and 128, dP at 256, dQ at 384.
  bool ok = true;

  if (warp == kSoftWarps) {
    if (lane == 0 && n > 0) {   // ------------------------------------------------ loads
      const uint64_t keep = ptx::policy_evict_last();
      ptx::mbar_arrive_expect_tx(&bars->res_full, 2 * C::kRes);
      const CUtensorMap* ma = kind == 0 ? &maps.kc : kind == 1 ? &maps.q : &maps.kb;
      const CUtensorMap* mb = kind == 0 ? &maps.vc : kind == 1 ? &maps.d_o : &maps.vb;
      const int slab = kind == 1 ? h : kvh, per = kind == 0 ? ctx : rows;
      for (int p = 0; p < PL; ++p)
        for (int s = 0; s < C::kSub; ++s) {
          const int y = (slab * PL + p) * per + tile * kRows;
          ptx::tma_load_2d(sm + (p * C::kSub + s) * C::kResTile, ma, &bars->res_full, 64 * s, y, keep);
          ptx::tma_load_2d(sm + C::kRes + (p * C::kSub + s) * C::kResTile, mb, &bars->res_full, 64 * s, y, keep);
        }
      int issued = 0;
      for (int i = 0; i < n && ok; ++i) {
        const int u = u0 + i, b = i % C::kStages;
        if (i >= C::kStages) ok = ptx::mbar_wait_sleep(&bars->freed[b], par(i - C::kStages), kBudget, pl.status);
        if (!ok) break;
        const CUtensorMap *m0, *m1;
        int slab_rows, sl, y0;
        if (kind == 1) {
          const bool own = u >= ctx_pieces;
          m0 = own ? &maps.kbs : &maps.kcs;
          m1 = own ? &maps.vbs : &maps.vcs;
          sl = kvh;
          slab_rows = own ? rows : ctx;
          y0 = own ? tile * kRows + (u - ctx_pieces) * C::kN : u * C::kN;
          ptx::mbar_arrive_expect_tx(&bars->full[b], 2 * C::kStr);
        } else {
          m0 = &maps.qs;
          m1 = &maps.d_os;
          sl = piece_head(u);
          slab_rows = rows;
          y0 = piece_row(u);
          ptx::mbar_arrive_expect_tx(&bars->full[b], 2 * C::kStr + C::kStat);
          float* st = stats(i);
          bulk_load(st, pl.lse2 + (size_t)sl * rows + y0, 4 * C::kN, &bars->full[b]);
          bulk_load(st + C::kN, pl.delta + (size_t)sl * rows + y0, 4 * C::kN, &bars->full[b]);
          bulk_load(st + 2 * C::kN, pl.row_anchor + y0, 4 * C::kN, &bars->full[b]);
        }
        uint8_t* dst = stage(i);
        for (int p = 0; p < PL; ++p)
          for (int s = 0; s < C::kSub; ++s) {
            const int y = (sl * PL + p) * slab_rows + y0;
            ptx::tma_load_2d(dst + (p * C::kSub + s) * C::kStrTile, m0, &bars->full[b], 64 * s, y, keep);
            ptx::tma_load_2d(dst + C::kStr + (p * C::kSub + s) * C::kStrTile, m1, &bars->full[b], 64 * s, y, keep);
          }
        issued = i + 1;
      }
      if (!ok) {   // a wait ran out: the copies in flight land before the CTA ends
        ptx::mbar_wait(&bars->res_full, 0, kBudget, nullptr);
        for (int i = max(0, issued - C::kStages); i < issued; ++i)
          ptx::mbar_wait(&bars->full[i % C::kStages], par(i), kBudget, nullptr);
      }
    }
  } else if (warp == kSoftWarps + 1) {
    if (lane == 0 && n > 0) {   // ------------------------------------------------ MMAs
      auto wait = [&](uint64_t* b, uint32_t p) {
        ok = ok && ptx::mbar_wait(b, p, kBudget, pl.status);
        ptx::tc_fence_after();
        return ok;
      };
      const uint8_t *ra = sm, *rb = sm + C::kRes;
      wait(&bars->res_full, 0);
      if (kind != 1) {
        const uint32_t tS = tA, tP = tA + 128, tV = tB, tK = tB + HD;
        // ra = K, rb = V; a stage holds Q, dO
        auto scores = [&](int i) {
          if (!wait(&bars->full[i % C::kStages], par(i))) return;
          mma_scores<HD, PL>(tS, ra, stage(i));
          ptx::mma_commit(&bars->s_full);
        };
        auto dprob = [&](int i) {
          mma_scores<HD, PL>(tP, rb, stage(i) + C::kStr);
          ptx::mma_commit(&bars->dp_full);
        };
        if (ok) scores(0);
        if (ok) dprob(0);
        for (int i = 0; i < n && ok; ++i) {
          if (!wait(&bars->p_ready, i & 1)) break;
          mma_gradient<HD, PL>(tV, tS, stage(i) + C::kStr, i > 0);
          if (C::kStages > 1 && i + 1 < n) {
            scores(i + 1);
            if (!ok) break;
          }
          if (!wait(&bars->ds_ready, i & 1)) break;
          mma_gradient<HD, PL>(tK, tP, stage(i), i > 0);
          ptx::mma_commit(&bars->freed[i % C::kStages]);
          if (i + 1 < n) {
            if (C::kStages == 1) scores(i + 1);
            if (ok) dprob(i + 1);
          }
        }
      } else {
        const uint32_t tP = tB, tQ = tB + 128;
        // ra = Q, rb = dO; a stage holds K, V
        auto scores = [&](int i) {
          if (!wait(&bars->full[i % C::kStages], par(i))) return;
          mma_scores<HD, PL>(tA + (i & 1) * 128, ra, stage(i));
        };
        auto dprob = [&](int i) {
          mma_scores<HD, PL>(tP, rb, stage(i) + C::kStr);
          ptx::mma_commit(&bars->s_full);
        };
        if (ok) scores(0);
        if (ok) dprob(0);
        for (int i = 0; i < n && ok; ++i) {
          if (C::kStages > 1 && i + 1 < n) {
            scores(i + 1);
            if (!ok) break;
          }
          if (!wait(&bars->p_ready, i & 1)) break;   // dP(i) is in registers
          if (C::kStages > 1 && i + 1 < n) dprob(i + 1);
          if (!wait(&bars->ds_ready, i & 1)) break;
          mma_gradient<HD, PL>(tQ, tA + (i & 1) * 128, stage(i), i > 0);
          ptx::mma_commit(&bars->freed[i % C::kStages]);
          if (C::kStages == 1 && i + 1 < n) {
            scores(i + 1);
            if (ok) dprob(i + 1);
          }
        }
      }
      ptx::mma_commit(&bars->done);
      if (!ok) ptx::mbar_wait(&bars->done, 0, kBudget, nullptr);   // what was issued ends before the CTA does
    }
  } else {   // ---------------------------------------------------------------------- softmax
    const int q4 = warp & 3, half = warp >> 2, me = 32 * q4 + lane;   // my lane of tensor memory
    const uint32_t lanes = static_cast<uint32_t>(32 * q4) << 16;
    const int c0 = half * C::kHalf;                                   // my first column
    const Scales sc = load_scales(pl.scale);
    const float sc2 = ldexpf(kLog2e * rsqrtf((float)HD), -sc.q - sc.k);   // the products' scales leave with it
    const float f_dp = ldexpf(1.f, sc.dp - sc.o - sc.v);
    const float scale = rsqrtf((float)HD);
    auto arrive = [&](uint64_t* b) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(b);
    };
    auto wait = [&](uint64_t* b, uint32_t p) {
      ok = ok && ptx::mbar_wait(b, p, kBudget, pl.status);
      ok = __all_sync(0xffffffffu, ok);
      ptx::tc_fence_after();
      return ok;
    };
    const int own = me / pl.block;            // block of my lane's row or key within its tile
    if (kind != 1) {
      const uint32_t tS = tA + lanes + c0, tP = tA + 128 + lanes + c0;
      const int key = tile * kRows + me;
      for (int i = 0; i < n; ++i) {
        if (!wait(&bars->full[i % C::kStages], par(i))) break;        // the rows' statistics
        const float* lse2 = stats(i) + c0;
        const float* delta = lse2 + C::kN;
        const int* anchor = reinterpret_cast<const int*>(lse2 + 2 * C::kN);
        const int r0 = piece_row(u0 + i) + c0 - (kind == 2 ? tile * kRows : 0);   // first row (within the tile: own keys)
        // rows below a boundary: only tiles that one crosses compare
        const bool compare = kind == 2 || reinterpret_cast<const int*>(stats(i) + 2 * C::kN)[0] < (tile + 1) * kRows;
        if (!wait(&bars->s_full, i & 1)) break;
        float p[C::kHalf];
#pragma unroll
        for (int c = 0; c < C::kHalf; c += 32) {
          ptx::tmem_ld32(tS + c, p + c);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 l = *reinterpret_cast<const float4*>(lse2 + c + j);
            p[c + j] = ex2(fmaf(p[c + j], sc2, -l.x));
            p[c + j + 1] = ex2(fmaf(p[c + j + 1], sc2, -l.y));
            p[c + j + 2] = ex2(fmaf(p[c + j + 2], sc2, -l.z));
            p[c + j + 3] = ex2(fmaf(p[c + j + 3], sc2, -l.w));
          }
          if (compare) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const bool seen = kind == 0 ? anchor[c + j] > key
                                          : static_cast<unsigned>(r0 + c + j - own * pl.block) < static_cast<unsigned>(pl.block);
              if (!seen) p[c + j] = 0.f;
            }
          }
          put_pairs<PL>(tS + c, p + c);
        }
        tmem_st_wait();
        arrive(&bars->p_ready);
        if (!wait(&bars->dp_full, i & 1)) break;
#pragma unroll
        for (int c = 0; c < C::kHalf; c += 32) {
          float d[32];
          ptx::tmem_ld32(tP + c, d);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 x = *reinterpret_cast<const float4*>(delta + c + j);
            d[j] = p[c + j] * fmaf(d[j], f_dp, -x.x);
            d[j + 1] = p[c + j + 1] * fmaf(d[j + 1], f_dp, -x.y);
            d[j + 2] = p[c + j + 2] * fmaf(d[j + 2], f_dp, -x.z);
            d[j + 3] = p[c + j + 3] * fmaf(d[j + 3], f_dp, -x.w);
          }
          put_pairs<PL>(tP + c, d);
        }
        tmem_st_wait();
        arrive(&bars->ds_ready);
      }
      // ---- dV and dK of my key, half of the columns each
      if (n > 0) wait(&bars->done, 0);
      if (ok) {
        const int e_v = -kPExp - sc.o, e_k = -kPExp - sc.dp - sc.q;
        constexpr int kCols = HD / 2;
        float* pk = nullptr;
        float* pv = nullptr;
        T* bk = nullptr;
        T* bv = nullptr;
        if (kind == 0) {
          if (key < pl.S) {
            const size_t o = (((size_t)h * pl.splits + split) * pl.S + key) * HD + half * kCols;
            pk = pl.dk_part + o;
            pv = pl.dv_part + o;
          }
        } else {
          const int at = tile * pl.per + own;
          if (own < pl.per && at < pl.N) {
            const size_t o = (((size_t)pl.order[at] * pl.block + (me - own * pl.block)) * pl.nkv + kvh) * HD + half * kCols;
            bk = static_cast<T*>(t.d_k_blk) + o;
            bv = static_cast<T*>(t.d_v_blk) + o;
          }
        }
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          float v[32] = {}, k[32] = {};
          if (n > 0) {
            ptx::tmem_ld32(tB + lanes + half * kCols + c, v);
            ptx::tmem_ld32(tB + lanes + HD + half * kCols + c, k);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            k[j] = ldexpf(k[j] * scale, e_k);
            v[j] = ldexpf(v[j], e_v);
          }
          if (pk) {
            store32(pk + c, k);
            store32(pv + c, v);
          }
          if (bk) {
            store32(bk + c, k);
            store32(bv + c, v);
          }
        }
      }
    } else {
      const uint32_t tP = tB + lanes + c0;
      const int r = tile * kRows + me;
      const float lse2 = pl.lse2[(size_t)h * rows + r], delta = pl.delta[(size_t)h * rows + r];
      const int anchor = pl.row_anchor[r];
      for (int i = 0; i < n; ++i) {
        if (!wait(&bars->s_full, i & 1)) break;
        const uint32_t tS = tA + (i & 1) * 128 + lanes + c0;
        // columns [first, first + count) of mine are seen
        int first = 0, count;
        if (i < ctx_pieces) {
          count = anchor - i * C::kN - c0;
        } else {
          first = own * pl.block - (i - ctx_pieces) * C::kN - c0;
          count = pl.block;
        }
        const bool all = __all_sync(0xffffffffu, i < ctx_pieces && count >= C::kHalf);
        float d[C::kHalf];
#pragma unroll
        for (int c = 0; c < C::kHalf; c += 32) ptx::tmem_ld32(tP + c, d + c);
        arrive(&bars->p_ready);   // dP may be overwritten
#pragma unroll
        for (int c = 0; c < C::kHalf; c += 32) {
          float s[32];
          ptx::tmem_ld32(tS + c, s);
#pragma unroll
          for (int j = 0; j < 32; ++j) s[j] = ex2(fmaf(s[j], sc2, -lse2)) * fmaf(d[c + j], f_dp, -delta);
          if (!all) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c + j < first || c + j >= first + count) s[j] = 0.f;
          }
          put_pairs<PL>(tS + c, s);
        }
        tmem_st_wait();
        arrive(&bars->ds_ready);
      }
      wait(&bars->done, 0);
      if (ok) {
        const int e_q = -kPExp - sc.dp - sc.k;
        constexpr int kCols = HD / 2;
        const int at = tile * pl.per + own;
        T* dst = nullptr;
        if (own < pl.per && at < pl.N)
          dst = static_cast<T*>(t.d_q) + (((size_t)pl.order[at] * pl.block + (me - own * pl.block)) * pl.nq + h) * HD +
                half * kCols;
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          float v[32];
          ptx::tmem_ld32(tB + 128 + lanes + half * kCols + c, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = ldexpf(v[j] * scale, e_q);
          if (dst) store32(dst + c, v);
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmem);
  }
}

// ---------------------------------------------------------------- context gradients from their shares
// d_k_ctx and d_v_ctx [S][nkv][hd]: the shares of a kv head's q heads and their
// splits, added in order; 4 values a thread.
template <typename T>
__global__ void __launch_bounds__(256) reduce_ctx_kernel(PackedBwdPlan pl, T* dk, T* dv) {
  griddep_wait();
  griddep_trigger();
  const int q = pl.hd / 4, shares = pl.nq / pl.nkv * pl.splits;
  const long long total = (long long)pl.S * pl.nkv * q;
  const size_t slab = (size_t)pl.S * pl.hd;
  for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < total; e += (long long)gridDim.x * 256) {
    const int d = (int)(e % q) * 4;
    const long long r = e / q;
    const int s = (int)(r % pl.S), h = (int)(r / pl.S);   // consecutive threads along a share's rows
    const size_t src = (size_t)h * shares * slab + (size_t)s * pl.hd + d;
    float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
    for (int i = 0; i < shares; ++i) {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(pl.dk_part + src + i * slab));
      const float4 b = __ldcs(reinterpret_cast<const float4*>(pl.dv_part + src + i * slab));
      k.x += a.x; k.y += a.y; k.z += a.z; k.w += a.w;
      v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
    }
    const size_t dst = ((size_t)s * pl.nkv + h) * pl.hd + d;
    auto put = [&](T* o, float4 x) {
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(o) = x;
      } else {
        __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
        *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
      }
    };
    put(dk + dst, k);
    put(dv + dst, v);
  }
}

// ---------------------------------------------------------------- lse of the forward
__global__ void __launch_bounds__(256) packed_lse_kernel(const float2* ml, int N, int block, int nq, int splits,
                                                         float* lse) {
  griddep_wait();
  griddep_trigger();
  const long long total = (long long)N * nq * block;
  for (long long r = (long long)blockIdx.x * 256 + threadIdx.x; r < total; r += (long long)gridDim.x * 256) {
    const float2* p = ml + r * splits;   // rows are ((n nq + h) block + i)
    float m = -3.0e38f, l = 0.f;
    for (int s = 0; s < splits; ++s)
      if (p[s].y > 0.f) m = fmaxf(m, p[s].x);
    for (int s = 0; s < splits; ++s)
      if (p[s].y > 0.f) l += p[s].y * expf(p[s].x - m);
    const int i = (int)(r % block), h = (int)(r / block % nq);
    const long long n = r / block / nq;
    lse[(n * block + i) * nq + h] = m + logf(l);
  }
}

size_t al(size_t v) { return (v + 255) & ~(size_t)255; }

template <typename T, int HD, int PL>
cudaError_t run_grad(const PackedBwdPlan& pl, const PackedBwdTensors& t, int sms, int* launches, cudaStream_t s) {
  using C = GradCfg<HD, PL>;
  const int rows = pl.T * kRows, ctx = pl.KT * kRows;
  cudaError_t e = launch_pdl(range_kernel<T, HD>, dim3((pl.N + kRangeThreads - 1) / kRangeThreads + pl.parts),
                             dim3(kRangeThreads), 0, s, pl, t);
  if (e != cudaSuccess) return e;
  ++*launches;
  const long long warps = (long long)rows * (pl.nq + pl.nkv) + (long long)ctx * pl.nkv;
  const int grid = (int)std::min<long long>((warps + 7) / 8, (long long)sms * 8);
  e = launch_pdl(pack_bwd_kernel<T, HD>, dim3(grid), dim3(256), 0, s, pl, t);
  if (e != cudaSuccess) return e;
  ++*launches;
  GradMaps m;
  const int q_rows = pl.nq * PL * rows, b_rows = pl.nkv * PL * rows, c_rows = pl.nkv * PL * std::max(ctx, kRows);
  auto enc = [&](CUtensorMap* a, CUtensorMap* b, const __half* p, int n) {   // a copy of 16-bit values, whatever they are
    return encode_activation_map(a, p, HD, n, HD, kRows) && encode_activation_map(b, p, HD, n, HD, C::kN);
  };
  if (!enc(&m.q, &m.qs, pl.q, q_rows) || !enc(&m.d_o, &m.d_os, pl.d_o, q_rows) || !enc(&m.kc, &m.kcs, pl.kc, c_rows) ||
      !enc(&m.vc, &m.vcs, pl.vc, c_rows) || !enc(&m.kb, &m.kbs, pl.kb, b_rows) || !enc(&m.vb, &m.vbs, pl.vb, b_rows))
    return cudaErrorInvalidValue;
  const int items = pl.KT * pl.nq * pl.splits + pl.T * pl.nq + pl.T * pl.nkv;
  e = launch_pdl(packed_grad_kernel<T, HD, PL>, dim3(items), dim3(kGradThreads), C::kBytes, s, pl, t, m);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (pl.S > 0) {
    const long long quads = (long long)pl.S * pl.nkv * (HD / 4);
    const int g = (int)std::min<long long>((quads + 255) / 256, (long long)sms * 16);
    e = launch_pdl(reduce_ctx_kernel<T>, dim3(g), dim3(256), 0, s, pl, static_cast<T*>(t.d_k_ctx),
                   static_cast<T*>(t.d_v_ctx));
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace

PackedBwdPlan packed_bwd_plan(void* ws, int N, int block, int S, int nq, int nkv, int hd, bool f32, int sms) {
  PackedBwdPlan p{};
  p.N = N;
  p.block = block;
  p.S = S;
  p.nq = nq;
  p.nkv = nkv;
  p.hd = hd;
  p.planes = f32 ? 2 : 1;
  p.per = kRows / block;
  p.T = (N + p.per - 1) / p.per;
  p.KT = (S + kRows - 1) / kRows;
  // enough context items to fill the GPU twice, at least one row tile each
  p.splits = std::max(1, std::min(p.T, (2 * sms + std::max(1, nq * p.KT) - 1) / std::max(1, nq * p.KT)));
  const size_t rows = (size_t)p.T * kRows, ctx = (size_t)std::max(p.KT, 1) * kRows;
  char* c = static_cast<char*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* r = ws ? c + at : nullptr;
    at += al(bytes);
    return r;
  };
  const size_t pe = 2 * (size_t)p.planes;
  p.status = reinterpret_cast<int32_t*>(take(4));
  p.parts = 2 * sms;
  p.part = reinterpret_cast<float*>(take(4 * (size_t)p.parts * kRangeValues));
  p.scale = reinterpret_cast<int32_t*>(take(4 * 5));
  p.order = reinterpret_cast<int32_t*>(take(4 * (size_t)N));
  p.sorted = reinterpret_cast<int32_t*>(take(4 * (size_t)N));
  p.row_anchor = reinterpret_cast<int32_t*>(take(4 * rows));
  p.lse2 = reinterpret_cast<float*>(take(4 * rows * nq));
  p.delta = reinterpret_cast<float*>(take(4 * rows * nq));
  p.q = reinterpret_cast<__half*>(take(pe * rows * nq * hd));
  p.d_o = reinterpret_cast<__half*>(take(pe * rows * nq * hd));
  p.kc = reinterpret_cast<__half*>(take(pe * ctx * nkv * hd));
  p.vc = reinterpret_cast<__half*>(take(pe * ctx * nkv * hd));
  p.kb = reinterpret_cast<__half*>(take(pe * rows * nkv * hd));
  p.vb = reinterpret_cast<__half*>(take(pe * rows * nkv * hd));
  const size_t part = 4 * (size_t)nq * p.splits * S * hd;
  p.dk_part = reinterpret_cast<float*>(take(part));
  p.dv_part = reinterpret_cast<float*>(take(part));
  p.bytes = at;
  return p;
}

cudaError_t packed_bwd_prepare(int hd, bool f32) {
  auto set = [](auto* k, int bytes) {
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  if (hd == 64)
    return f32 ? set(packed_grad_kernel<float, 64, 2>, GradCfg<64, 2>::kBytes)
               : set(packed_grad_kernel<__nv_bfloat16, 64, 1>, GradCfg<64, 1>::kBytes);
  return f32 ? set(packed_grad_kernel<float, 128, 2>, GradCfg<128, 2>::kBytes)
             : set(packed_grad_kernel<__nv_bfloat16, 128, 1>, GradCfg<128, 1>::kBytes);
}

cudaError_t packed_bwd_run(const PackedBwdPlan& pl, const PackedBwdTensors& t, int sms, int* launches, cudaStream_t s) {
  *launches = 0;
  if (pl.hd == 64)
    return pl.planes == 2 ? run_grad<float, 64, 2>(pl, t, sms, launches, s)
                          : run_grad<__nv_bfloat16, 64, 1>(pl, t, sms, launches, s);
  return pl.planes == 2 ? run_grad<float, 128, 2>(pl, t, sms, launches, s)
                        : run_grad<__nv_bfloat16, 128, 1>(pl, t, sms, launches, s);
}

cudaError_t packed_lse_launch(const float2* ml, int N, int block, int nq, int splits, float* lse, cudaStream_t s) {
  const long long rows = (long long)N * nq * block;
  const int grid = (int)std::min<long long>((rows + 255) / 256, 4096);
  return launch_pdl(packed_lse_kernel, dim3(grid), dim3(256), 0, s, ml, N, block, nq, splits, lse);
}

}  // namespace dflash
