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
//   context keys  (kv head, 128 keys, share): for each row tile that sees them,
//                 of every head in turn, S' = K Q', dP' = V dO' (keys on the
//                 tensor-memory lanes), dV += P' dO, dK += dS' Q, with P' and dS'
//                 written back to tensor memory as the A operand; where several
//                 CTAs share a key tile's work their sums go to memory as fp32 and
//                 a last kernel adds them in order;
//   rows          (q head, 128 rows): for each key tile S = Q K', dP = dO V',
//                 dQ += dS K;
//   own keys      (kv head, row tile): as context keys, over the tile's own rows.
// S and dP are thus computed twice (7 products instead of 5), and nothing is
// accumulated with atomics: the results do not change from run to run.  dQ beside
// dK and dV would need a second sum of 128 x hd in tensor memory for each row tile
// that a key tile meets, or 2 GB of fp32 atomics (at the training shape below).
//
// Measured (512 blocks of 16 in 4,096 positions, 32 query and 8 kv heads of 128,
// bf16): 866 us, of which the ranges take 45 (HBM, 5.6 TB/s), the layout 87 (HBM,
// 6.6 TB/s), the gradients 692 and the shares' sum 12; 693 GFLOP of five products
// at 0.80 PFLOP/s, the gradient kernel's seven at 1.40 PFLOP/s.  What bounds
// that kernel is the hand-over between tensor cores and softmax warps: a tile of
// context keys takes about 2,800 cycles, 2,050 of them MMAs.  100 blocks of 10 in
// 1,999 positions: 111 us; 12 blocks of 8 in 500: 23 us, four launches' latency.
//
// In a CTA one thread loads tiles by TMA, one issues the MMAs, and sixteen warps
// turn S and dP into P and dS.  The MMA thread alternates so that the tensor
// cores work on the other product while the warps work on one:
//   keys:  dV(i) S(i+1) | dK(i) dP(i+1)      rows:  S(i+1) dP(i+1) dQ(i)
// Each operand tile is staged once and read in both directions: K-major for S and
// dP, MN-major as the B operand of the gradients.
//
// Operands, P and dS enter the products as fp16, which has three more bits than
// bf16, scaled by powers of two so that its range holds them: q, k, v and d_out
// each by the power that brings its largest value to 2^14 .. 2^15, P (at most 1) by
// 2^14, and ds by what the largest norms of d_out's and v's rows allow it
// (|dp| <= |d_out_r| |v_j|; for dQ, whose sums are one row's, by the row's own
// norm of d_out).  The scales are folded into factors that are there
// anyway, and powers of two are exact.  bf16 tensors take one plane: the operands
// are then exact but for d_out, and d_out, P and ds are rounded by 2^-12 of
// themselves, an eighth of the rounding of the bf16 gradients.  fp32 tensors
// take each operand, P and ds included, as a hi + lo pair (22 bits) and each
// product as three MMAs (hi hi, hi lo, lo hi).  Every sum and the softmax are fp32;
// the tensor cores' sums truncate (by 2e-8 a step of 16 rows, measured, all to the
// same side), so those of fp32 tensors are kept short: a context item moves them to
// its share's memory every 96 steps.  512 blocks of 16 in 4,096 positions, 32/8 heads:
// 3.04 ms with heads of 128 and 1.50 with 64.  Never moved: 2.85 ms, but an error of
// 1.6e-5 of the gradients' norm instead of 2.4e-6 (200 blocks in 3,000); a share in
// memory for every 8 tiles instead: 3.49 ms and 2.1 GB of them.
#include <cuda.h>

#include <algorithm>
#include <climits>

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
constexpr int kRowExpMax = 40;       // more than d_out's fp16 can tell a row from zero
constexpr int kRangeValues = 6;      // largest |q|, |k|, |v|, |d_out|, and largest norm of a row of v, d_out
constexpr int kRangeThreads = 512;

// Exponents e of the scales 2^e of q, k, v and d_out, and of dp (and D):
// ds is held as P 2^14 (dp - D) 2^dp.
struct Scales {
  int q, k, v, o, dp;
};
__device__ __forceinline__ float pow2(int e) { return ldexpf(1.f, e); }
// v 2^e in two exact steps, each within fp32's range.
struct Pow2 {
  float a, b;
  __device__ __forceinline__ explicit Pow2(int e) : a(pow2(e / 2)), b(pow2(e - e / 2)) {}
  __device__ __forceinline__ float operator()(float v) const { return v * a * b; }
};
// The exponent that brings m into [2^14, 2^15), within what a float holds.
__device__ __forceinline__ int scale_exp(float m) {
  if (!(m > 0.f) || isinf(m)) return 0;
  return max(-120, min(120, kOpExp - ilogbf(m)));
}
// The e with n < 2^e.
__device__ __forceinline__ int norm_exp(float n) { return n > 0.f && !isinf(n) ? ilogbf(n) + 1 : 0; }
__device__ __forceinline__ Scales scales_of(const float* m) {
  Scales s;
  s.q = scale_exp(m[0]);
  s.k = scale_exp(m[1]);
  s.v = scale_exp(m[2]);
  s.o = scale_exp(m[3]);
  // |dp - D| <= 2 |d_out| |v| by the rows' norms
  s.dp = -(norm_exp(m[4]) + norm_exp(m[5]) + 1);
  return s;
}
__device__ __forceinline__ Scales load_scales(const int32_t* p) { return Scales{p[0], p[1], p[2], p[3], p[4]}; }

// ---------------------------------------------------------------- loads
__device__ __forceinline__ void unpack16(uint4 r, float* v, float) {
  v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack16(uint4 r, float* v, __nv_bfloat16) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}
__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// The 16 bytes at p; `aligned`: whether its tensor starts on a 16-byte boundary.
template <typename T>
__device__ __forceinline__ uint4 load16(const T* p, bool aligned) {
  if (aligned) return *reinterpret_cast<const uint4*>(p);
  constexpr int E = 16 / sizeof(T);
  alignas(16) T v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = p[e];
  return *reinterpret_cast<const uint4*>(v);
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

// Largest value (and, where NORM, largest norm of a row) of `rows` rows of HD
// values.  A warp has eight 16-byte loads a lane in flight; the eight sums of
// squares are reduced together, half of them handed to the other lanes at each
// step.
template <typename T, int HD, bool NORM>
__device__ __forceinline__ void range_rows(const T* x, long long rows, int part, int parts, float& mx, float& nm) {
  constexpr int E = 16 / sizeof(T), L = HD / E, U = 8;   // values of a load, lanes of a row
  constexpr int kRowsPer = 32 / L * U;
  const int lane = threadIdx.x & 31, sub = lane / L, col = lane % L * E;
  const bool aligned = aligned16(x);
  const long long step = (long long)parts * (kRangeThreads / 32) * kRowsPer;
  for (long long r0 = ((long long)part * (kRangeThreads / 32) + (threadIdx.x >> 5)) * kRowsPer; r0 < rows; r0 += step) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * (32 / L) + sub;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (r < rows) raw[u] = load16(x + (size_t)r * HD + col, aligned);
    }
    float sq[U];
    bool odd = false;   // a square may have left fp32's range
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[E];
      unpack16(raw[u], v, T());
      sq[u] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        mx = fmaxf(mx, fabsf(v[e]));
        if (NORM) sq[u] = fmaf(v[e], v[e], sq[u]);
      }
      if (NORM) odd |= !(sq[u] < 1.0e36f) || (sq[u] < 1.0e-30f && (raw[u].x | raw[u].y | raw[u].z | raw[u].w) != 0);
    }
    if (NORM) {
      int n = U;
#pragma unroll
      for (int o = L / 2; o; o >>= 1) {
        if (n > 1) {
          n /= 2;
#pragma unroll
          for (int j = 0; j < U / 2; ++j)
            if (j < n) {
              const bool up = lane & o;
              const float keep = up ? sq[j + n] : sq[j], send = up ? sq[j] : sq[j + n];
              sq[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        } else {
          sq[0] += __shfl_xor_sync(0xffffffffu, sq[0], o);
        }
      }
      if (!__any_sync(0xffffffffu, odd)) {   // (every row's sum is in some lane; n is 1 for all shapes: L >= 8)
        nm = fmaxf(nm, sqrtf(sq[0]));
      } else {   // each row over its largest value
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float v[E], m = 0.f, s2 = 0.f;
          unpack16(raw[u], v, T());
#pragma unroll
          for (int e = 0; e < E; ++e) m = fmaxf(m, fabsf(v[e]));
          for (int o = L / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
          for (int e = 0; e < E; ++e) s2 = m > 0.f ? fmaf(v[e] / m, v[e] / m, s2) : 0.f;
          for (int o = L / 2; o; o >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
          nm = fmaxf(nm, m * sqrtf(s2));
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
  // context rows that no block sees are not read, whatever they hold
  __shared__ int s_seen[kRangeThreads / 32];
  int seen = 0;
  for (int n = threadIdx.x; n < pl.N; n += kRangeThreads) seen = max(seen, t.anchors[n]);
  seen = __reduce_max_sync(0xffffffffu, min(seen, pl.S));
  if ((threadIdx.x & 31) == 0) s_seen[threadIdx.x >> 5] = seen;
  const long long qr = (long long)pl.N * pl.block * pl.nq, br = (long long)pl.N * pl.block * pl.nkv;
  range_rows<T, HD, false>(static_cast<const T*>(t.q), qr, part, parts, m[0], none);
  range_rows<float, HD, true>(t.d_out, qr, part, parts, m[3], m[5]);
  range_rows<T, HD, false>(static_cast<const T*>(t.k_blk), br, part, parts, m[1], none);
  range_rows<T, HD, true>(static_cast<const T*>(t.v_blk), br, part, parts, m[2], m[4]);
  __syncthreads();
  seen = __reduce_max_sync(0xffffffffu, s_seen[threadIdx.x % (kRangeThreads / 32)]);
  const long long cr = (long long)seen * pl.nkv;
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
// Eight values of a lane from 16 bytes of T (bf16) or 32 (fp32).
template <typename T>
struct Values8 {
  uint4 raw[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, bool aligned) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) raw[i] = load16(p + i * (16 / sizeof(T)), aligned);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) raw[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) unpack16(raw[i], v + i * (16 / (int)sizeof(T)), T());
  }
};

// Eight values times `scale` as one or two fp16 planes `plane` apart; v becomes
// what the planes hold.
template <int PL>
__device__ __forceinline__ void put_planes(__half* dst, size_t plane, float scale, float* v) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float x = v[2 * j] * scale, y = v[2 * j + 1] * scale;
    const __half2 a = __floats2half2_rn(x, y);
    h[j] = *reinterpret_cast<const uint32_t*>(&a);
    float2 f = __half22float2(a);
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
    if (PL == 2) {
      const __half2 b = __floats2half2_rn(x - f.x, y - f.y);
      l[j] = *reinterpret_cast<const uint32_t*>(&b);
      f = __half22float2(b);
      v[2 * j] += f.x;
      v[2 * j + 1] += f.y;
    }
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
  if (PL == 2) *reinterpret_cast<uint4*>(dst + plane) = make_uint4(l[0], l[1], l[2], l[3]);
}

// A warp takes a few heads of a row at a time (32 * 8 / hd of them side by side,
// kPackUnroll times): query rows (with D and lse), then the blocks' own keys and
// values, then the context's.  Bound by HBM: q, out and d_out are read once.
constexpr int kPackUnroll = 2;
template <int HD> __host__ __device__ constexpr int pack_heads() { return 256 / HD * kPackUnroll; }

template <typename T, int HD, int PL>
__global__ void __launch_bounds__(256) pack_bwd_kernel(PackedBwdPlan pl, PackedBwdTensors t) {
  griddep_wait();
  griddep_trigger();
  constexpr int L = HD / 8, R = 32 / L, U = kPackUnroll, H = pack_heads<HD>();
  const int lane = threadIdx.x & 31, sub = lane / L, col = lane % L * 8;
  const int g = pl.block, rows = pl.T * kRows, ctx = pl.KT * kRows;
  const int q_groups = (pl.nq + H - 1) / H, k_groups = (pl.nkv + H - 1) / H;
  const long long n_q = (long long)rows * q_groups, n_b = (long long)rows * k_groups, n_c = (long long)ctx * k_groups;
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
  // Each key tile's first row tile whose last block is anchored behind the tile's
  // first key, and first one whose first block is anchored behind all its keys.
  for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < pl.KT; j += gridDim.x * blockDim.x) {
    int lo = 0, hi = pl.T;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (pl.sorted[min((mid + 1) * pl.per, pl.N) - 1] > j * kRows) hi = mid; else lo = mid + 1;
    }
    const int first = lo;
    for (hi = pl.T; lo < hi;) {
      const int mid = (lo + hi) >> 1;
      if (pl.sorted[mid * pl.per] >= (j + 1) * kRows) hi = mid; else lo = mid + 1;
    }
    pl.seen_by[j] = make_int2(first, lo);
  }
  const int seen = pl.N ? pl.sorted[pl.N - 1] : 0;   // context rows that some block sees
  const float f_q = pow2(s_sc.q), f_k = pow2(s_sc.k), f_v = pow2(s_sc.v), f_o = pow2(s_sc.o);
  const int e_d = s_sc.dp - s_sc.o;   // D is summed over the scaled d_out
  const int e_o = norm_exp(s_max[5]) + s_sc.o;   // |d_out_r| 2^o < 2^e_o
  const bool al_q = aligned16(t.q), al_g = aligned16(t.d_out), al_o = aligned16(t.out);
  // block and position of a row; -1: padding
  auto place = [&](int r, int& n, int& i) {
    const int k = r % kRows, b = k / g, at = (r / kRows) * pl.per + b;
    n = b < pl.per && at < pl.N ? pl.order[at] : -1;
    i = k - b * g;
    return at;
  };
  for (long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < n_q + n_b + n_c; w += warps) {
    if (w < n_q) {
      const int r = (int)(w / q_groups), h0 = (int)(w - (long long)r * q_groups) * H + sub;
      int n, i;
      const int at = place(r, n, i);
      const size_t row = ((size_t)(n < 0 ? 0 : n) * g + i) * pl.nq;
      Values8<T> q[U];
      Values8<float> go[U], oo[U];
      float l[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * R;
        if (n >= 0 && h < pl.nq) {
          const size_t o = (row + h) * HD + col;
          q[u].load(static_cast<const T*>(t.q) + o, al_q);
          go[u].load(t.d_out + o, al_g);
          oo[u].load(t.out + o, al_o);
          l[u] = fmaf(t.lse[row + h], kLog2e, -(float)kPExp);
        } else {
          q[u].zero();
          go[u].zero();
          oo[u].zero();
          l[u] = INFINITY;
        }
      }
      float d[U], n2[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * R;
        float a[8], b[8], c[8];
        q[u].get(a);
        go[u].get(b);
        oo[u].get(c);
        d[u] = n2[u] = 0.f;
        if (h < pl.nq) {
          const size_t dst = ((size_t)h * PL * rows + r) * HD + col, plane = (size_t)rows * HD;
          put_planes<PL>(pl.q + dst, plane, f_q, a);
          put_planes<PL>(pl.d_o + dst, plane, f_o, b);
          // D from d_out as the products see it: its rounding then cancels in dp - D as exactly as d_out itself would
#pragma unroll
          for (int e = 0; e < 8; ++e) d[u] = fmaf(b[e], c[e], d[u]), n2[u] = fmaf(b[e], b[e], n2[u]);
        }
      }
#pragma unroll
      for (int o = L / 2; o; o >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          d[u] += __shfl_xor_sync(0xffffffffu, d[u], o);
          n2[u] += __shfl_xor_sync(0xffffffffu, n2[u], o);
        }
      if (col == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = h0 + u * R;
          if (h < pl.nq) {
            pl.lse2[(size_t)h * rows + r] = l[u];
            pl.delta[(size_t)h * rows + r] = ldexpf(d[u], e_d);
            // |d_out_r| 2^o < 2^(floor(log2(n2) / 2) + 1)
            const int below = n2[u] > 0.f ? e_o - (ilogbf(n2[u]) >> 1) - 1 : 0;
            pl.row_scale[(size_t)h * rows + r] = pow2(max(0, min(kRowExpMax, below)));
            if (h == 0) pl.row_anchor[r] = n >= 0 ? pl.sorted[at] : INT_MAX;
          }
        }
      }
    } else {
      const bool blk = w < n_q + n_b;
      const long long x = blk ? w - n_q : w - n_q - n_b;
      const int r = (int)(x / k_groups), h0 = (int)(x - (long long)r * k_groups) * H + sub, slab = blk ? rows : ctx;
      long long row = -1;   // of [tokens][nkv]
      if (blk) {
        int n, i;
        place(r, n, i);
        if (n >= 0) row = ((long long)n * g + i) * pl.nkv;
      } else if (r < seen) {
        row = (long long)r * pl.nkv;
      }
      const T* k = static_cast<const T*>(blk ? t.k_blk : t.k_ctx);
      const T* v = static_cast<const T*>(blk ? t.v_blk : t.v_ctx);
      const bool al_k = aligned16(k), al_v = aligned16(v);
      Values8<T> ks[U], vs[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * R;
        if (row >= 0 && h < pl.nkv) {
          ks[u].load(k + (size_t)(row + h) * HD + col, al_k);
          vs[u].load(v + (size_t)(row + h) * HD + col, al_v);
        } else {
          ks[u].zero();
          vs[u].zero();
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * R;
        float a[8], b[8];
        ks[u].get(a);
        vs[u].get(b);
        if (h < pl.nkv) {
          const size_t dst = ((size_t)h * PL * slab + r) * HD + col, plane = (size_t)slab * HD;
          put_planes<PL>((blk ? pl.kb : pl.kc) + dst, plane, f_k, a);
          put_planes<PL>((blk ? pl.vb : pl.vc) + dst, plane, f_v, b);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- tensor-core pieces
// Shared-memory descriptors (128-byte swizzle, tiles of rows of 64 fp16): the
// low word holds the address, which a step through the tile is added to, the
// high word is the same for all: 8 rows are 1024 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// K-major: a row's values run along K.
__device__ __forceinline__ uint32_t desc_k(const void* tile) { return (ptx::smem_u32(tile) >> 4) | (1u << 16); }
// MN-major: a row's 64 values run along N, the rows along K; lbo: bytes to the
// tile of the next 64 values.
__device__ __forceinline__ uint32_t desc_mn(const void* tile, uint32_t lbo) {
  return (ptx::smem_u32(tile) >> 4) | ((lbo >> 4) << 16);
}
// Instruction descriptor, kind::f16: fp16 A and B (formats zero), fp32 D, M x N, both K-major.
constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t kBMajorMN = 1u << 16;

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
// D[tmem] (+)= A[smem] B[smem]'
__device__ __forceinline__ void mma_smem(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]: A's rows on the lanes, two consecutive K values
// to a 32-bit column.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// C (16 or 32) consecutive columns of this warp's lanes; tmem_ld_wait before use.
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r) {
  if constexpr (C == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  }
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// The values of a load, tied to the wait so that no use moves before it.
template <int C>
__device__ __forceinline__ void tmem_values(const uint32_t* r, float* v) {
#pragma unroll
  for (int i = 0; i < C; ++i) {
    uint32_t x = r[i];
    asm volatile("" : "+r"(x));
    v[i] = __uint_as_float(x);
  }
}
template <int C>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t* v) {
  if constexpr (C == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
  } else {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  }
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Box (x = column, y = row) of a tensor map into shared memory.  No cache
// hint: the operands are read again and again, but exceed what L2 can keep.
__device__ __forceinline__ void tma_tile(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                   ptx::smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   ptx::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(ptx::smem_u32(src)), "r"(bytes)
               : "memory");
}
// Until this thread's stores have left shared memory.
__device__ __forceinline__ void bulk_store_wait() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 values at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)), "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}

__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }
// Zero but for columns [from, to) of C.
template <int C>
__device__ __forceinline__ void keep_columns(float* v, int from, int to) {
  const uint32_t below = from <= 0 ? 0u : from >= 32 ? ~0u : (1u << from) - 1;
  const uint32_t bits = (to <= 0 ? 0u : to >= 32 ? ~0u : (1u << to) - 1) & ~below;
#pragma unroll
  for (int j = 0; j < C; ++j)
    if (!(bits >> j & 1)) v[j] = 0.f;
}
// C values as C / 2 registers of fp16 pairs.
template <int C>
__device__ __forceinline__ void pairs_of(const float* v, uint32_t* h) {
#pragma unroll
  for (int j = 0; j < C / 2; ++j) h[j] = as_u32(__floats2half2_rn(v[2 * j], v[2 * j + 1]));
}
// The pairs into C / 2 columns from `at` on and, with two planes, the values'
// rounding residuals into the next C / 2: the C columns that the values were read
// from.
template <int PL, int C>
__device__ __forceinline__ void put_pairs(uint32_t at, const uint32_t* h, const float* v) {
  tmem_st<C / 2>(at, h);
  if (PL == 2) {
    uint32_t l[C / 2];
#pragma unroll
    for (int j = 0; j < C / 2; ++j) {
      const float2 f = __half22float2(as_half2(h[j]));
      l[j] = as_u32(__floats2half2_rn(v[2 * j] - f.x, v[2 * j + 1] - f.y));
    }
    tmem_st<C / 2>(at + C / 2, l);
  }
}

// ---------------------------------------------------------------- the gradient kernel
// Warps 0..15 softmax (warp w: lanes 32 (w % 4), a quarter w / 4 of the columns),
// warp 16 loads, warp 17 issues the MMAs.
constexpr int kSoftWarps = 16;
constexpr int kParts = kSoftWarps / 4;             // warps of a lane quarter
// 96 registers a thread, the most that five warps of one scheduler leave each other.
// ptxas spills 52 bytes (bf16, heads of 128), 28 (of 64), 44 and 316 (fp32).
constexpr int kGradThreads = 32 * (kSoftWarps + 2);

// Two streams of tiles pass the two resident operands: the first feeds S and dK
// (or dQ), the second dP and dV.  The first one's tiles are needed soonest and
// freed last, so it has one stage more.
template <int HD, int PL>
struct GradCfg {
  static constexpr int kSub = HD / 64;
  static constexpr int kN = PL == 2 && HD == 128 ? 64 : 128;   // rows of a streamed tile
  static constexpr int kS0 = PL == 2 && HD == 128 ? 2 : 3;
  static constexpr int kS1 = kS0 - 1;
  static constexpr int kResTile = kRows * 128;             // 128 rows x 64 values
  static constexpr int kRes = PL * kSub * kResTile;        // one resident operand
  static constexpr int kStrTile = kN * 128;
  static constexpr int kStr = PL * kSub * kStrTile;        // one streamed tile
  static constexpr int kStat = kN * 4;                     // lse2 with the first stream, delta with the second
  static constexpr int kOff0 = 2 * kRes;
  static constexpr int kOff1 = kOff0 + kS0 * kStr;
  static constexpr int kOffStat = kOff1 + kS1 * kStr;
  static constexpr int kOffBars = kOffStat + (kS0 + kS1) * kStat;
  static constexpr int kUsed = kOffBars + 160;
  // more than half of an SM's shared memory: the CTA takes all of tensor memory
  static constexpr int kBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static constexpr int kCols = kN / kParts;                // columns of S of one softmax warp
  static constexpr int kPitch = HD * 4 + 16;               // fp32 rows staged on their way out: no bank conflicts
  // tensor memory.  Keys: S at 0, dP at 128, dV at 256, dK behind it.  Rows: S in
  // two buffers at 0 and kN, dP behind them, dQ behind that.  With two planes the
  // small products (hi lo and lo hi) have sums of their own where there is room, kLo
  // columns further (0: none): the tensor cores truncate a sum at each step, and so
  // the large one takes a third of the steps.
  static constexpr int kColP = 128, kColV = 256, kColK = kColV + HD, kLoKeys = PL == 2 && HD == 64 ? 2 * HD : 0;
  static constexpr int kColPRows = 2 * kN, kColQ = kN == 64 ? 256 : 384, kLoRows = PL == 2 ? HD : 0;
  // Two planes: streamed tiles after which a context item moves its sums to memory
  // and starts them again, 96 truncating steps of 16 rows (8 a tile with heads of 64,
  // whose small products have sums of their own, 12 with 128).
  static constexpr int kDrain = HD == 64 ? 12 : 8;
  static constexpr uint32_t kTmem = 512;
  static_assert(kColK + kLoKeys + HD <= 512 && kColQ + kLoRows + HD <= 512 && kColPRows + kN <= kColQ, "tensor memory");
  static_assert(kBytes <= 227 * 1024 && 2 * kRows * kPitch <= kOffStat, "shared memory");
};

// A barrier's waiters have to look at a phase before the next but one
// completes.  Keys: what completes phase i + 1 of s_full, dp_full, p_ready and
// ds_ready waits, through the MMA thread or the warps, for every waiter of
// phase i.  A stage of the first stream is loaded again after dK, that is after
// all warps have left it (ds_ready); the tile of one of the second, which MMAs
// alone read, after dV, but its delta, which the warps read, after dK too: its
// phase completes only then.
// Rows: S and dP of tile i + 1 wait for the warps' loads of tile i (p_ready) and
// not for their dS, so ds_ready alternates between two barriers.
struct GradBars {
  uint64_t res_full, full0[3], freed0[3], full1[2], freed1[2], s_full, dp_full, p_ready, ds_ready[2], done;
  uint32_t tmem;
};

struct GradMaps {
  CUtensorMap q, d_o, kc, vc, kb, vb;         // boxes of 64 values x 128 rows (resident)
  CUtensorMap qs, d_os, kcs, vcs, kbs, vbs;   // x kN rows (streamed)
};

// CTAs that share the n streamed tiles of one context key tile.
__device__ __forceinline__ int shares_of(const PackedBwdPlan& pl, int n) { return (n + pl.share - 1) / pl.share; }

// S (+)= A B' over hd: A 128 resident rows, B kN streamed rows, both K-major.
// With two planes the small products come first, while the sum is small.
template <int HD, int PL>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t res, uint32_t str) {
  using C = GradCfg<HD, PL>;
  constexpr uint32_t id = idesc_f16(kRows, C::kN);
  uint32_t acc = 0;
#pragma unroll
  for (int pr = (PL == 2 ? 0 : 2); pr < 3; ++pr) {   // hi lo, lo hi, hi hi
    const int pa = pr == 1, pb = pr == 0;
#pragma unroll
    for (int s = 0; s < C::kSub; ++s)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        mma_smem(d, res + ((pa * C::kSub + s) * C::kResTile >> 4) + 2 * k,
                 str + ((pb * C::kSub + s) * C::kStrTile >> 4) + 2 * k, id, acc);
        acc = 1;
      }
  }
}
// G (+)= A B: A the P or dS of 128 lanes in tensor memory (columns of `a` as
// put_pairs left them), B kN streamed rows read along their values.  LO: columns
// from G to its sum of small products.
template <int HD, int PL, int LO>
__device__ __forceinline__ void mma_gradient(uint32_t d, uint32_t a, uint32_t str, uint32_t accumulate) {
  using C = GradCfg<HD, PL>;
  constexpr uint32_t id = idesc_f16(kRows, HD) | kBMajorMN;
  uint32_t acc = accumulate;
#pragma unroll
  for (int pr = (PL == 2 ? 0 : 2); pr < 3; ++pr) {
    const int pa = pr == 1, pb = pr == 0;
    if (LO && pr == 2) acc = accumulate;
#pragma unroll
    for (int k = 0; k < C::kN / 16; ++k) {
      const int chunk = 16 * k / C::kCols, in = 16 * k % C::kCols;
      mma_tmem(LO && pr < 2 ? d + LO : d, a + chunk * C::kCols + pa * (C::kCols / 2) + in / 2,
               str + (pb * C::kSub * C::kStrTile >> 4) + k * (2048 >> 4), id, acc);
      acc = 1;
    }
  }
}

// 32 columns of a gradient in tensor memory, with the small products' sum `lo`
// columns further (0: none).
__device__ __forceinline__ void read_sum(uint32_t at, int lo, float* v) {
  uint32_t raw[32];
  tmem_ld<32>(at, raw);
  tmem_ld_wait();
  tmem_values<32>(raw, v);
  if (lo) {
    float small[32];
    tmem_ld<32>(at + lo, raw);
    tmem_ld_wait();
    tmem_values<32>(raw, small);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += small[j];
  }
}
// A key's gradients of a share while its item still runs: [hd / 4][128 keys][4], so
// that a warp's accesses are consecutive.  `d` is the thread's place of 32 columns;
// each thread meets its own values only.
__device__ __forceinline__ void add_so_far(const float4* d, float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float4 b = __ldcg(d + j * kRows);
    v[4 * j] += b.x, v[4 * j + 1] += b.y, v[4 * j + 2] += b.z, v[4 * j + 3] += b.w;
  }
}
// dK and dV of this thread's key (columns `at` and `at` - HD of tensor memory) into
// dk and dv in memory.  The warps of a lane quarter take the 32-column groups of
// both in turn.  A call, so that its registers are not the main loop's.
template <int HD, int LO>
__device__ __noinline__ void drain_sums(uint32_t at, float4* dk, float4* dv, int part, float to_k, float to_k2, float to_v,
                                        float to_v2, bool fresh) {
  constexpr int kGroups = HD / 32;
#pragma unroll 1
  for (int gq = part; gq < 2 * kGroups; gq += kParts) {
    const int m = gq / kGroups, c = gq % kGroups * 32;   // 0: dK, 1: dV
    float v[32];
    read_sum(at - m * HD + c, LO, v);
    const float a = m ? to_v : to_k, b = m ? to_v2 : to_k2;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = v[j] * a * b;
    float4* d = (m ? dv : dk) + c / 4 * kRows;
    if (!fresh) add_so_far(d, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) __stcg(d + j * kRows, make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
  }
}

template <typename T, int HD, int PL>
__global__ void __launch_bounds__(kGradThreads, 1) packed_grad_kernel(const __grid_constant__ PackedBwdPlan pl,
                                                                      const __grid_constant__ PackedBwdTensors t,
                                                                      const __grid_constant__ GradMaps maps) {
  using C = GradCfg<HD, PL>;
  extern __shared__ __align__(1024) uint8_t sm[];
  GradBars* bars = reinterpret_cast<GradBars*>(sm + C::kOffBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  griddep_trigger();
  if (ptx::smem_u32(sm) & 1023) {   // the swizzled tiles need it; no device places shared memory otherwise
    if (tid == 0) report_status(pl.status, DFLASH_ERR_UNSUPPORTED);
    return;
  }

  // ---- this CTA's item
  const int G = pl.nq / pl.nkv, rows = pl.T * kRows, ctx = pl.KT * kRows;
  constexpr int kPer = kRows / C::kN;        // streamed tiles of 128 rows
  const int n_ctx = pl.KT * pl.nkv * pl.splits, n_own = pl.T * pl.nkv;
  int kind, h, tile, share = 0;              // kind 0: context keys, 1: rows, 2: own keys (h: kv head unless 1)
  int u0 = 0, u1, first = 0, whole = 0;      // streamed tiles [u0, u1)
  {
    int b = blockIdx.x;
    if (b < n_ctx) {
      // the first keys are seen by most: longest items first.  Streamed: the
      // row tiles from `first` on (from `whole` on they see every key), head by head
      kind = 0;
      tile = b / (pl.nkv * pl.splits);
      b -= tile * pl.nkv * pl.splits;
      h = b / pl.splits;
      share = b - h * pl.splits;
      const int2 seen = pl.seen_by[tile];
      first = seen.x;
      whole = seen.y;
      const int n = (pl.T - first) * kPer * G, shares = shares_of(pl, n);
      if (share >= shares) return;
      u0 = (int)((long long)n * share / shares);
      u1 = (int)((long long)n * (share + 1) / shares);
    } else if (b >= n_ctx + n_own) {
      // streamed: the context below the tile's largest anchor (`first` tiles), then
      // the tile's own keys.  The shortest items end the launch.
      kind = 1;
      b -= n_ctx + n_own;
      tile = pl.T - 1 - b / pl.nq;
      h = b % pl.nq;
      first = (pl.sorted[min((tile + 1) * pl.per, pl.N) - 1] + C::kN - 1) / C::kN;
      u1 = first + kPer;
    } else {
      // streamed: the row tile, head by head
      kind = 2;
      b -= n_ctx;
      tile = b / pl.nkv;
      h = b % pl.nkv;
      u1 = G * kPer;
    }
  }
  const int kvh = kind == 1 ? h / G : h, n = u1 - u0;
  // head and first row of streamed tile u (kinds 0 and 2)
  const int per_head = kind == 0 ? (pl.T - first) * kPer : kPer, row0 = (kind == 0 ? first : tile) * kRows;

  if (tid == 0) {
    ptx::mbar_init(&bars->res_full, 1);
    for (int s = 0; s < C::kS0; ++s) {
      ptx::mbar_init(&bars->full0[s], 1);
      ptx::mbar_init(&bars->freed0[s], 1);
    }
    for (int s = 0; s < C::kS1; ++s) {
      ptx::mbar_init(&bars->full1[s], 1);
      ptx::mbar_init(&bars->freed1[s], 1);
    }
    ptx::mbar_init(&bars->s_full, 1);
    ptx::mbar_init(&bars->dp_full, 1);
    ptx::mbar_init(&bars->ds_ready[0], kSoftWarps);
    ptx::mbar_init(&bars->ds_ready[1], kSoftWarps);
    ptx::mbar_init(&bars->p_ready, kSoftWarps);
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

  auto str0 = [&](int i) { return sm + C::kOff0 + (i % C::kS0) * C::kStr; };
  auto str1 = [&](int i) { return sm + C::kOff1 + (i % C::kS1) * C::kStr; };
  auto lse_of = [&](int i) { return sm + C::kOffStat + (i % C::kS0) * C::kStat; };
  auto delta_of = [&](int i) { return sm + C::kOffStat + (C::kS0 + i % C::kS1) * C::kStat; };
  auto par0 = [](int i) { return static_cast<uint32_t>(i / C::kS0) & 1u; };
  auto par1 = [](int i) { return static_cast<uint32_t>(i / C::kS1) & 1u; };
  bool ok = true;

  if (warp == kSoftWarps) {
    if (lane == 0) {   // ------------------------------------------------ loads
      {
        ptx::mbar_arrive_expect_tx(&bars->res_full, 2 * C::kRes);
        const CUtensorMap* ma = kind == 0 ? &maps.kc : kind == 1 ? &maps.q : &maps.kb;
        const CUtensorMap* mb = kind == 0 ? &maps.vc : kind == 1 ? &maps.d_o : &maps.vb;
        for (int p = 0; p < PL; ++p)
          for (int s = 0; s < C::kSub; ++s) {
            const int y = (h * PL + p) * (kind == 0 ? ctx : rows) + tile * kRows;
            tma_tile(sm + (p * C::kSub + s) * C::kResTile, ma, &bars->res_full, 64 * s, y);
            tma_tile(sm + C::kRes + (p * C::kSub + s) * C::kResTile, mb, &bars->res_full, 64 * s, y);
          }
      }
      int i0 = 0, i1 = 0;   // tiles issued of each stream
      for (int i = 0; i < n && ok; ++i) {
        const int u = u0 + i;
        const CUtensorMap *m0 = &maps.qs, *m1 = &maps.d_os;
        int slab, slab_rows = rows, y0;
        if (kind == 1) {
          const bool own = u >= first;
          m0 = own ? &maps.kbs : &maps.kcs;
          m1 = own ? &maps.vbs : &maps.vcs;
          slab = kvh;
          slab_rows = own ? rows : ctx;
          y0 = own ? tile * kRows + (u - first) * C::kN : u * C::kN;
        } else {
          const int hh = u / per_head;
          slab = h * G + hh;
          y0 = row0 + (u - hh * per_head) * C::kN;
        }
        auto issue = [&](uint8_t* dst, const CUtensorMap* m, uint64_t* bar) {
          for (int p = 0; p < PL; ++p)
            for (int s = 0; s < C::kSub; ++s)
              tma_tile(dst + (p * C::kSub + s) * C::kStrTile, m, bar, 64 * s, (slab * PL + p) * slab_rows + y0);
        };
        if (i >= C::kS0) ok = ptx::mbar_wait_sleep(&bars->freed0[i % C::kS0], par0(i - C::kS0), kBudget, pl.status);
        if (!ok) break;
        uint64_t* bar = &bars->full0[i % C::kS0];
        ptx::mbar_arrive_expect_tx(bar, C::kStr + (kind == 1 ? 0 : C::kStat));
        issue(str0(i), m0, bar);
        if (kind != 1) bulk_load(lse_of(i), pl.lse2 + (size_t)slab * rows + y0, C::kStat, bar);
        i0 = i + 1;
        if (i >= C::kS1) ok = ptx::mbar_wait_sleep(&bars->freed1[i % C::kS1], par1(i - C::kS1), kBudget, pl.status);
        if (!ok) break;
        bar = &bars->full1[i % C::kS1];
        ptx::mbar_arrive_expect_tx(bar, C::kStr + (kind == 1 ? 0 : C::kStat));
        issue(str1(i), m1, bar);
        i1 = i + 1;
        if (kind != 1) {
          const int j = i - C::kS1;   // the last tile whose delta was there
          if (j >= 0) ok = ptx::mbar_wait_sleep(&bars->freed0[j % C::kS0], par0(j), kBudget, pl.status);
          if (!ok) break;
          bulk_load(delta_of(i), pl.delta + (size_t)slab * rows + y0, C::kStat, bar);
        }
      }
      if (!ok) {   // a wait ran out: the copies in flight land before the CTA ends
        ptx::mbar_wait(&bars->res_full, 0, kBudget, nullptr);
        for (int i = max(0, i0 - C::kS0); i < i0; ++i) ptx::mbar_wait(&bars->full0[i % C::kS0], par0(i), kBudget, nullptr);
        for (int i = max(0, i1 - C::kS1); i < i1; ++i)   // (the last may wait for a delta that was not sent)
          ptx::mbar_wait(&bars->full1[i % C::kS1], par1(i), kBudget / 8, nullptr);
      }
    }
  } else if (warp == kSoftWarps + 1) {
    // ------------------------------------------------ MMAs
    // The whole warp runs this, so that what it computes is uniform; one elected
    // lane issues each group of MMAs with the commits behind it.
    auto wait = [&](uint64_t* b, uint32_t p) {
      if (!__all_sync(0xffffffffu, ptx::mbar_try_wait(b, p))) {
        ok = ok && ptx::mbar_wait(b, p, kBudget, pl.status);
        ok = __all_sync(0xffffffffu, ok);
      }
      ptx::tc_fence_after();
      return ok;
    };
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t ra = desc_k(sm), rb = desc_k(sm + C::kRes);
    const uint32_t k0 = desc_k(sm + C::kOff0), k1 = desc_k(sm + C::kOff1);
    const uint32_t g0 = desc_mn(sm + C::kOff0, C::kStrTile), g1 = desc_mn(sm + C::kOff1, C::kStrTile);
    constexpr uint32_t kStep = C::kStr >> 4;
    // a stage of each stream: this tile's, and the next one's with its phase
    int s0 = 0, s1 = 0, n0 = 0, n1 = 0;
    uint32_t ph0 = 0, ph1 = 0;
    auto wait2 = [&](uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb) {
      const bool x = ptx::mbar_try_wait(a, pa), y = ptx::mbar_try_wait(b, pb);
      if (__all_sync(0xffffffffu, x && y)) {
        ptx::tc_fence_after();
        return ok;
      }
      return wait(a, pa) && wait(b, pb);
    };
    auto arrived0 = [&] { return wait(&bars->full0[n0], ph0); };
    auto arrived1 = [&] { return wait(&bars->full1[n1], ph1); };
    auto next0 = [&] { if (++n0 == C::kS0) n0 = 0, ph0 ^= 1; };
    auto next1 = [&] { if (++n1 == C::kS1) n1 = 0, ph1 ^= 1; };
    // The next tiles are waited for before what the warps are still at, so that
    // the MMAs of both products go out together (with a single stage the next
    // tile of the second stream comes only after dV).
    constexpr bool kAhead = C::kS1 > 1;
    if (wait(&bars->res_full, 0) && arrived0() && arrived1()) {
      if (kind != 1) {
        // resident K, V; streamed Q, dO
        const uint32_t tS = tm, tP = tm + C::kColP, tV = tm + C::kColV, tK = tm + C::kColK;
        if (elect()) {
          mma_scores<HD, PL>(tS, ra, k0);
          ptx::mma_commit(&bars->s_full);
          mma_scores<HD, PL>(tP, rb, k1);
          ptx::mma_commit(&bars->dp_full);
        }
        __syncwarp();
        next0();
        next1();
        for (int i = 0; i < n; ++i) {
          const bool more = i + 1 < n;
          // (sums start again where the warps have moved them to memory, which p_ready says)
          const uint32_t go_on = (PL == 2 && kind == 0 ? i % C::kDrain : i) != 0;
          if (more ? !wait2(&bars->full0[n0], ph0, &bars->p_ready, i & 1) : !wait(&bars->p_ready, i & 1)) break;
          if (elect()) {
            mma_gradient<HD, PL, C::kLoKeys>(tV, tS, g1 + s1 * kStep, go_on);
            ptx::mma_commit(&bars->freed1[s1]);
            if (more) {
              mma_scores<HD, PL>(tS, ra, k0 + n0 * kStep);
              ptx::mma_commit(&bars->s_full);
            }
          }
          __syncwarp();
          if (more && kAhead ? !wait2(&bars->full1[n1], ph1, &bars->ds_ready[0], i & 1) : !wait(&bars->ds_ready[0], i & 1)) break;
          if (elect()) {
            mma_gradient<HD, PL, C::kLoKeys>(tK, tP, g0 + s0 * kStep, go_on);
            ptx::mma_commit(&bars->freed0[s0]);
          }
          __syncwarp();
          if (more) {
            if (!kAhead && !arrived1()) break;
            if (elect()) {
              mma_scores<HD, PL>(tP, rb, k1 + n1 * kStep);
              ptx::mma_commit(&bars->dp_full);
            }
            __syncwarp();
          }
          s0 = n0;
          s1 = n1;
          next0();
          next1();
        }
      } else {
        // resident Q, dO; streamed K, V
        const uint32_t tP = tm + C::kColPRows;
        if (elect()) {
          mma_scores<HD, PL>(tm, ra, k0);
          mma_scores<HD, PL>(tP, rb, k1);
          ptx::mma_commit(&bars->s_full);
          ptx::mma_commit(&bars->freed1[0]);
        }
        __syncwarp();
        next0();
        next1();
        for (int i = 0; i < n; ++i) {
          const bool more = i + 1 < n;
          // (S goes over dS(i - 1), which the last dQ has taken, dP over dP(i) once it is in registers)
          if (more ? !wait2(&bars->full0[n0], ph0, &bars->full1[n1], ph1) : false) break;
          if (!wait(&bars->p_ready, i & 1)) break;
          if (more) {
            if (elect()) {
              mma_scores<HD, PL>(tm + (~i & 1) * C::kN, ra, k0 + n0 * kStep);
              mma_scores<HD, PL>(tP, rb, k1 + n1 * kStep);
              ptx::mma_commit(&bars->s_full);
              ptx::mma_commit(&bars->freed1[n1]);
            }
            __syncwarp();
          }
          if (!wait(&bars->ds_ready[i & 1], (i >> 1) & 1)) break;
          if (elect()) {
            mma_gradient<HD, PL, C::kLoRows>(tm + C::kColQ, tm + (i & 1) * C::kN, g0 + s0 * kStep, i > 0);
            ptx::mma_commit(&bars->freed0[s0]);
          }
          __syncwarp();
          s0 = n0;
          s1 = n1;
          next0();
          next1();
        }
      }
    }
    if (elect()) ptx::mma_commit(&bars->done);
    __syncwarp();
    if (!ok) ptx::mbar_wait(&bars->done, 0, kBudget, nullptr);   // what was issued ends before the CTA does
  } else {   // ---------------------------------------------------------------------- softmax
    constexpr int NC = C::kCols;
    const int q4 = warp & 3, part = warp >> 2, me = 32 * q4 + lane;   // my lane of tensor memory
    const uint32_t lanes = static_cast<uint32_t>(32 * q4) << 16;
    const int c0 = part * NC;                                         // my first column
    const Scales sc = load_scales(pl.scale);
    const float scale = rsqrtf((float)HD);
    const float sc2 = ldexpf(kLog2e * scale, -sc.q - sc.k);   // the products' scales leave with it
    const float f_dp = ldexpf(1.f, sc.dp - sc.o - sc.v);
    auto arrive = [&](uint64_t* b) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(b);
    };
    auto wait = [&](uint64_t* b, uint32_t p) {
      if (!__all_sync(0xffffffffu, ptx::mbar_try_wait(b, p))) {
        ok = ok && ptx::mbar_wait(b, p, kBudget, pl.status);
        ok = __all_sync(0xffffffffu, ok);
      }
      ptx::tc_fence_after();
      return ok;
    };
    const int own = me / pl.block;            // block of my lane's row or key within its tile
    // staged output rows: matrix m's row r at m * kRows * kPitch + r * kPitch
    auto stage32 = [&](int m, int c, const float* v, bool wide) {   // 32 columns from c on
      uint8_t* d = sm + (size_t)(m * kRows + me) * C::kPitch + c * (wide ? 4 : (int)sizeof(T));
      if (wide || sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(d + 4 * j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 b = __floats2bfloat162_rn(v[j + 2 * i], v[j + 2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t*>(&b);
          }
          *reinterpret_cast<uint4*>(d + 2 * j) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    };
    // All rows staged, the first 128 threads send matrix 0's, the next 128 matrix
    // 1's.  Every warp comes here, after a timeout too: the barrier needs them all.
    auto send = [&](void* dst, uint32_t bytes) {
      ptx::fence_proxy_async_shared();
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory");
      if (dst) {
        bulk_store(dst, sm + (size_t)tid * C::kPitch, bytes);
        bulk_store_wait();
      }
    };
    // place of a tile's row r in [N][block][heads][hd], or nullptr in padding
    auto block_row = [&](void* base, int r, int heads, int head) -> void* {
      const int b = r / pl.block, at = tile * pl.per + b;
      if (b >= pl.per || at >= pl.N) return nullptr;
      return static_cast<T*>(base) + (((size_t)pl.order[at] * pl.block + (r - b * pl.block)) * heads + head) * HD;
    };
    constexpr int kGroups = HD / 32;          // 32-column groups of a gradient row
    if (kind != 1) {
      const uint32_t tS = tmem + lanes + c0, tP = tS + C::kColP;
      const int key = tile * kRows + me;
      int in_head = u0 % per_head;            // streamed tile within its head
      int s0 = 0, s1 = 0;                     // stages of the two streams and their phases
      uint32_t ph0 = 0, ph1 = 0;
      // The columns' lse2 and delta are read ahead, while the warps wait for S and
      // dP: MMAs with both operands in shared memory take its whole bandwidth,
      // and a load in the middle of the arithmetic waits for them.
      float4 st[NC / 4];
      auto load_stats = [&](int slot) {
        const float4* x = reinterpret_cast<const float4*>(sm + C::kOffStat + slot * C::kStat) + c0 / 4;
#pragma unroll
        for (int j = 0; j < NC / 4; ++j) st[j] = x[j];
      };
      auto so_far = [&](float* base) {   // my key's place in this share's rows
        return reinterpret_cast<float4*>(base + (((size_t)h * pl.splits + share) * ctx + tile * kRows) * HD) + me;
      };
      int i = 0;
      for (;;) {
        const int end = PL == 2 && kind == 0 ? min(n, i + C::kDrain) : n;
        if (wait(&bars->full0[s0], ph0)) load_stats(s0);
        for (; i < end; ++i) {
          const int r0 = row0 + in_head * C::kN + c0;   // my first column's row
          const bool compare = kind == 2 || r0 < whole * kRows;
          if (++in_head == per_head) in_head = 0;
          if (!wait(&bars->s_full, i & 1)) break;
          const int anchor = kind == 0 && compare ? __ldg(pl.row_anchor + r0 + lane % NC) : 0;   // of column `lane`
          // P: as the fp16 pairs that enter dV and, with two planes, as fp32
          uint32_t pairs[NC / 2];
          float p[NC];
          {
            uint32_t raw[NC];
            tmem_ld<NC>(tS, raw);
            tmem_ld_wait();
            tmem_values<NC>(raw, p);
          }
#pragma unroll
          for (int j = 0; j < NC; j += 4) {
            const float4 l = st[j / 4];
            const float2 a = fma2(make_float2(p[j], p[j + 1]), make_float2(sc2, sc2), make_float2(-l.x, -l.y));
            const float2 b = fma2(make_float2(p[j + 2], p[j + 3]), make_float2(sc2, sc2), make_float2(-l.z, -l.w));
            p[j] = ex2(a.x);
            p[j + 1] = ex2(a.y);
            p[j + 2] = ex2(b.x);
            p[j + 3] = ex2(b.y);
          }
          if (compare) {
            int from = own * pl.block - (r0 - row0), to = from + pl.block;   // own keys: my block's rows
            if (kind == 0) {   // the rows from the first one anchored behind my key on (anchors ascend)
              from = 0;
              to = NC;
#pragma unroll 1
              for (int step = NC / 2; step; step /= 2)
                if (__shfl_sync(0xffffffffu, anchor, from + step - 1) <= key) from += step;
              if (__shfl_sync(0xffffffffu, anchor, from) <= key) ++from;
            }
            keep_columns<NC>(p, from, to);
          }
          pairs_of<NC>(p, pairs);
          put_pairs<PL, NC>(tS, pairs, p);
          tmem_st_wait();
          arrive(&bars->p_ready);
          if (!wait(&bars->full1[s1], ph1)) break;
          load_stats(C::kS0 + s1);
          if (++s1 == C::kS1) s1 = 0, ph1 ^= 1;
          if (!wait(&bars->dp_full, i & 1)) break;
          uint32_t hi[NC / 2];
          float d[NC];
          {
            uint32_t raw[NC];
            tmem_ld<NC>(tP, raw);
            tmem_ld_wait();
            tmem_values<NC>(raw, d);
          }
          const float2 f = make_float2(f_dp, f_dp);
#pragma unroll
          for (int j = 0; j < NC; j += 4) {
            const float4 x = st[j / 4];
            const float2 a = fma2(make_float2(d[j], d[j + 1]), f, make_float2(-x.x, -x.y));
            const float2 b = fma2(make_float2(d[j + 2], d[j + 3]), f, make_float2(-x.z, -x.w));
            if (PL == 1) {
              // P 2^14 from its pairs, dp - D (at most 1) in fp32 until their product is rounded: as fp16 it would be
              // 0 below 2^-25, and blocks of small d_out would lose what the 2^14 gives them.  (P kept in fp32 instead
              // spills: 1,393 us for the training shape, 860 so.)
              const float2 u = mul2(__half22float2(as_half2(pairs[j / 2])), a);
              const float2 v = mul2(__half22float2(as_half2(pairs[j / 2 + 1])), b);
              hi[j / 2] = as_u32(__floats2half2_rn(u.x, u.y));
              hi[j / 2 + 1] = as_u32(__floats2half2_rn(v.x, v.y));
            } else {
              const float2 u = mul2(make_float2(p[j], p[j + 1]), a), v = mul2(make_float2(p[j + 2], p[j + 3]), b);
              d[j] = u.x, d[j + 1] = u.y, d[j + 2] = v.x, d[j + 3] = v.y;
            }
          }
          if (PL == 2) pairs_of<NC>(d, hi);
          put_pairs<PL, NC>(tP, hi, d);
          tmem_st_wait();
          arrive(&bars->ds_ready[0]);
          if (++s0 == C::kS0) s0 = 0, ph0 ^= 1;
          if (i + 1 < end) {
            if (!wait(&bars->full0[s0], ph0)) break;
            load_stats(s0);
          }
        }
        if (PL == 1 || !ok || i == n) break;
        // dK(i - 1) is the last to add to the sums.  (Its stage's phase before that one has completed: tile i - 1,
        // which the warps have seen, was loaded after it.)
        if (!wait(&bars->freed0[(i - 1) % C::kS0], par0(i - 1))) break;
        const Pow2 to_v(-kPExp - sc.o), to_k(-kPExp - sc.dp - sc.q);
        drain_sums<HD, C::kLoKeys>(tmem + lanes + C::kColK, so_far(pl.dk_part), so_far(pl.dv_part), part, to_k.a * scale,
                                   to_k.b, to_v.a, to_v.b, i == C::kDrain);
      }
      // ---- dV and dK of my key: the warps of a lane quarter take the 32-column groups of both in turn
      wait(&bars->done, 0);
      const bool drained = PL == 2 && kind == 0 && n > C::kDrain;
      if (ok) {
        const Pow2 to_v(-kPExp - sc.o), to_k(-kPExp - sc.dp - sc.q);
#pragma unroll
        for (int x = 0; x < 2 * kGroups / kParts; ++x) {
          const int gq = x * kParts + part, m = gq / kGroups, c = gq % kGroups * 32;   // matrix 0: dK, 1: dV
          float v[32];
          read_sum(tmem + lanes + (m ? C::kColV : C::kColK) + c, C::kLoKeys, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = m ? to_v(v[j]) : to_k(v[j] * scale);
          if (drained) add_so_far(so_far(m ? pl.dv_part : pl.dk_part) + c / 4 * kRows, v);
          stage32(m, c, v, kind == 0);
        }
      }
      if (drained) ptx::fence_proxy_async_global();   // the rows go where the sums so far were
      void* dst = nullptr;
      if (ok && tid < 2 * kRows) {
        const int r = tid % kRows;
        const bool v = tid >= kRows;
        if (kind == 0) {
          if (tile * kRows + r < pl.S)
            dst = (v ? pl.dv_part : pl.dk_part) + (((size_t)h * pl.splits + share) * ctx + tile * kRows + r) * HD;
        } else {
          dst = block_row(v ? t.d_v_blk : t.d_k_blk, r, pl.nkv, kvh);
        }
      }
      send(dst, HD * (kind == 0 ? 4 : (int)sizeof(T)));
    } else {
      const int r = tile * kRows + me;
      // dQ's sums are a row's own, and so is the scale of its ds: rows of small d_out keep their bits
      const float up = pl.row_scale[(size_t)h * rows + r], f_row = f_dp * up;
      const float lse2 = pl.lse2[(size_t)h * rows + r], delta = pl.delta[(size_t)h * rows + r] * up;
      const int anchor = pl.row_anchor[r];
      for (int i = 0; i < n; ++i) {
        if (!wait(&bars->s_full, i & 1)) break;
        const uint32_t tS = tmem + lanes + (i & 1) * C::kN + c0;
        // columns [from, from + count) of mine are seen
        int from = 0, count;
        if (i < first) {
          count = anchor - i * C::kN - c0;
        } else {
          from = own * pl.block - (i - first) * C::kN - c0;
          count = pl.block;
        }
        const bool all = __all_sync(0xffffffffu, i < first && count >= NC);
        float d[NC], s[NC];
        {
          uint32_t raw[NC], raw2[NC];
          tmem_ld<NC>(tmem + lanes + C::kColPRows + c0, raw);
          tmem_ld<NC>(tS, raw2);
          tmem_ld_wait();
          tmem_values<NC>(raw, d);
          tmem_values<NC>(raw2, s);
        }
        arrive(&bars->p_ready);   // dP may be overwritten
#pragma unroll
        for (int j = 0; j < NC; j += 2) {
          const float2 a = fma2(make_float2(s[j], s[j + 1]), make_float2(sc2, sc2), make_float2(-lse2, -lse2));
          const float2 b = fma2(make_float2(d[j], d[j + 1]), make_float2(f_row, f_row), make_float2(-delta, -delta));
          const float2 x = mul2(make_float2(ex2(a.x), ex2(a.y)), b);
          s[j] = x.x;
          s[j + 1] = x.y;
        }
        if (!all) keep_columns<NC>(s, from, from + count);
        uint32_t hi[NC / 2];
        pairs_of<NC>(s, hi);
        put_pairs<PL, NC>(tS, hi, s);
        tmem_st_wait();
        arrive(&bars->ds_ready[i & 1]);
      }
      wait(&bars->done, 0);
      if (ok) {
        const Pow2 to_q(-kPExp - sc.dp - sc.k);
        const float down = scale / up;
#pragma unroll
        for (int c = part * 32; c < HD; c += kParts * 32) {
          float v[32];
          read_sum(tmem + lanes + C::kColQ + c, C::kLoRows, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = to_q(v[j] * down);
          stage32(0, c, v, false);
        }
      }
      send(ok && tid < kRows ? block_row(t.d_q, tid, pl.nq, h) : nullptr, HD * (int)sizeof(T));
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
// d_k_ctx and d_v_ctx [S][nkv][hd]: a key tile's shares added in order, 4
// values a thread.  grid (key tiles x parts of a tile, kv heads).
template <typename T, int HD, int PL>
__global__ void __launch_bounds__(256) reduce_ctx_kernel(PackedBwdPlan pl, T* dk, T* dv) {
  griddep_wait();
  griddep_trigger();
  constexpr int Q = HD / 4, kParts = kRows * Q / 256;
  const int tile = blockIdx.x / kParts, h = blockIdx.y;
  __shared__ int s_shares;
  if (threadIdx.x == 0)
    s_shares = shares_of(pl, (pl.T - pl.seen_by[tile].x) * (kRows / GradCfg<HD, PL>::kN) * (pl.nq / pl.nkv));
  __syncthreads();
  const int shares = s_shares, e = blockIdx.x % kParts * 256 + threadIdx.x;
  const int s = tile * kRows + e / Q, d = e % Q * 4;
  if (s >= pl.S) return;
  const size_t slab = (size_t)pl.KT * kRows * HD, src = (size_t)h * pl.splits * slab + (size_t)s * HD + d;
  float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
  for (int i = 0; i < shares; ++i) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(pl.dk_part + src + i * slab));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(pl.dv_part + src + i * slab));
    k.x += a.x; k.y += a.y; k.z += a.z; k.w += a.w;
    v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
  }
  const size_t dst = ((size_t)s * pl.nkv + h) * HD + d;
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
  auto heads = [](int n) { return (n + pack_heads<HD>() - 1) / pack_heads<HD>(); };
  const long long warps = (long long)rows * (heads(pl.nq) + heads(pl.nkv)) + (long long)ctx * heads(pl.nkv);
  const int grid = (int)std::min<long long>((warps + 7) / 8, (long long)sms * 8);
  e = launch_pdl(pack_bwd_kernel<T, HD, PL>, dim3(grid), dim3(256), 0, s, pl, t);
  if (e != cudaSuccess) return e;
  ++*launches;
  GradMaps m;
  const int q_rows = pl.nq * PL * rows, b_rows = pl.nkv * PL * rows, c_rows = pl.nkv * PL * std::max(ctx, kRows);
  auto enc = [&](CUtensorMap* a, CUtensorMap* b, const __half* p, int n) {   // a copy of 16-bit values, whatever they are
    if (!encode_activation_map(a, p, HD, n, HD, kRows)) return false;
    if (C::kN != kRows) return encode_activation_map(b, p, HD, n, HD, C::kN);
    *b = *a;
    return true;
  };
  if (!enc(&m.q, &m.qs, pl.q, q_rows) || !enc(&m.d_o, &m.d_os, pl.d_o, q_rows) || !enc(&m.kc, &m.kcs, pl.kc, c_rows) ||
      !enc(&m.vc, &m.vcs, pl.vc, c_rows) || !enc(&m.kb, &m.kbs, pl.kb, b_rows) || !enc(&m.vb, &m.vbs, pl.vb, b_rows))
    return cudaErrorInvalidValue;
  const int items = pl.KT * pl.nkv * pl.splits + pl.T * pl.nq + pl.T * pl.nkv;
  e = launch_pdl(packed_grad_kernel<T, HD, PL>, dim3(items), dim3(kGradThreads), C::kBytes, s, pl, t, m);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (pl.S > 0) {
    e = launch_pdl(reduce_ctx_kernel<T, HD, PL>, dim3(pl.KT * (kRows * HD / 4 / 256), pl.nkv), dim3(256), 0, s, pl,
                   static_cast<T*>(t.d_k_ctx), static_cast<T*>(t.d_v_ctx));
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
  // Streamed tiles of one context item.  An item costs about as much as three
  // tiles before and after them, and its sums a trip through memory, so items are
  // long where there are enough of them to go round: `all` tiles for the first key
  // tile, half as many on average, half an item an SM.  (Cases of 16 x 8 and 32 x 8
  // key tiles and kv heads: 7 -> 135 and 1231 us, 18 -> 114 and 1002, 36 -> 109 and
  // 926, 128 -> 109 and 876; of 8 x 2: 3 -> 32 us, 12 -> 53.)
  const int per = kRows / (f32 && hd == 128 ? GradCfg<128, 2>::kN : kRows);
  const long long all = (long long)(nq / nkv) * p.T * per;
  // Each share has its own rows in memory, so no more of them than make about eight
  // items an SM: that memory follows the SM count and the context, not the blocks
  // (4,096 blocks of 16 in 32,768 positions, 32/8 heads of 128: 0.27 GB; shares of 128
  // tiles would take 4.3).  It costs no time: that case takes 38.6 ms in bf16 (44.9 with
  // shares of 128), 1,024 blocks in 8,192 2.77 (2.78).
  const long long tiles = std::max(1LL, (long long)p.KT * nkv), most = (8LL * sms + tiles - 1) / tiles;
  p.share = (int)std::max({3LL, std::min(128LL, all * p.KT * nkv / sms), (all + most - 1) / most});
  p.splits = (int)((all + p.share - 1) / p.share);
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
  p.parts = sms;   // one CTA of the range kernel an SM
  p.part = reinterpret_cast<float*>(take(4 * (size_t)p.parts * kRangeValues));
  p.scale = reinterpret_cast<int32_t*>(take(4 * 5));
  p.order = reinterpret_cast<int32_t*>(take(4 * (size_t)N));
  p.sorted = reinterpret_cast<int32_t*>(take(4 * (size_t)N));
  p.seen_by = reinterpret_cast<int2*>(take(8 * (size_t)std::max(p.KT, 1)));
  p.row_anchor = reinterpret_cast<int32_t*>(take(4 * rows));
  p.lse2 = reinterpret_cast<float*>(take(4 * rows * nq));
  p.delta = reinterpret_cast<float*>(take(4 * rows * nq));
  p.row_scale = reinterpret_cast<float*>(take(4 * rows * nq));
  p.q = reinterpret_cast<__half*>(take(pe * rows * nq * hd));
  p.d_o = reinterpret_cast<__half*>(take(pe * rows * nq * hd));
  p.kc = reinterpret_cast<__half*>(take(pe * ctx * nkv * hd));
  p.vc = reinterpret_cast<__half*>(take(pe * ctx * nkv * hd));
  p.kb = reinterpret_cast<__half*>(take(pe * rows * nkv * hd));
  p.vb = reinterpret_cast<__half*>(take(pe * rows * nkv * hd));
  const size_t part = 4 * (size_t)nkv * p.splits * p.KT * kRows * hd;
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
