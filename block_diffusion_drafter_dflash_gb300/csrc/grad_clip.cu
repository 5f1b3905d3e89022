// Global gradient norm over many tensors, and clipping (the training recipe
// of the paper, section 7.1, clips at 1.0):
//
//   norm = sqrt(sum_i g_i^2)     out_i = g_i * min(1, max_norm / norm)
//
// Two kernels over the same list of tensors.  The first reads every gradient
// once; the second reads and writes them, walking the list backwards so that
// what the first read last is still in L2 (129 MB; a drafter's few megabytes
// stay there altogether).  Both are bound by HBM: 1.05 G bf16 gradients (an
// 8B-shaped drafter's five layers and fusion) take 296 us for the norm (7.1 TB/s) and 660 us
// to scale (6.4 TB/s of reads and writes); 1.9 M fp32 ones 9.5 us in all, two
// launches' latency.
//
// The list travels in the launch's parameters (up to kMaxTensors a launch,
// longer lists take several launches): no table in device memory, so a call
// can be captured into a graph and the caller keeps nothing alive.  A tensor
// is cut into chunks of kChunkVec 16-byte vectors; chunk c goes to CTA c mod
// grid, found by binary search over the tensors' first chunks.
//
// Sums.  A thread squares and adds its vectors of one chunk in fp32 (at most
// 64 values), then adds that to its running sum in double; the CTAs' sums are
// added in double in a fixed order, so the result does not change from run to
// run.  Where the fp32 sum leaves the range in which no square overflowed or
// vanished, the values, still in registers, are squared again in double:
// gradients of 1e30 or 1e-30 have a finite, non-zero norm.
//
// A norm that is not finite (some gradient is infinite or NaN) leaves the
// gradients as they are, and so does one within the limit (bit for bit).
#include <cmath>

#include "common.cuh"
#include "grad_clip.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                          // vectors of a thread and chunk
constexpr int kChunkVec = kThreads * kVec;       // 32 KB
// Tensors a launch's parameters hold: 2 KB or 16 KB of them
constexpr int kFewTensors = 64, kMaxTensors = 512;
constexpr int kCtasPerSm = 4;

struct Entry {
  const void* in;
  void* out;
  long long numel;
  long long first;   // number of its first chunk, shifted left by one, plus 1 if bf16
};
template <int MAX>
struct Table {
  static constexpr int kMax = MAX;
  int n;
  long long chunks;
  Entry e[MAX];
};

// Entry holding chunk c.
template <class Tab>
__device__ __forceinline__ int find_entry(const Tab& t, long long c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((t.e[mid].first >> 1) <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// This thread's vectors of chunk c: word offsets and what of them lies inside
// the tensor.  Vectors are aligned to 16 bytes of the input; the first and the
// last of a tensor may be partly outside.
struct Piece {
  const char* base;    // the input's address, rounded down to 16 bytes
  long long v0;        // this thread's first vector
  long long nvec;      // vectors of the tensor
  long long lo, hi;    // bytes [lo, hi) from base belong to the tensor
};
__device__ __forceinline__ Piece piece(const Entry& e, long long c) {
  Piece p;
  const uintptr_t a = reinterpret_cast<uintptr_t>(e.in);
  p.base = reinterpret_cast<const char*>(a & ~uintptr_t(15));
  p.lo = (long long)(a & 15);
  p.hi = p.lo + e.numel * (e.first & 1 ? 2 : 4);
  p.nvec = (p.hi + 15) >> 4;
  p.v0 = (c - (e.first >> 1)) * kChunkVec + threadIdx.x;
  return p;
}
// Vector v of the piece; bytes outside the tensor read as zero, without a load.
template <bool LAST>
__device__ __forceinline__ uint4 load_vec(const Piece& p, long long v, bool bf16) {
  const long long b = v << 4;
  if (b >= p.lo && b + 16 <= p.hi) {
    const uint4* q = reinterpret_cast<const uint4*>(p.base + b);
    return LAST ? __ldcs(q) : *q;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const long long o = b + 2 * j;
    if (bf16) {
      if (o >= p.lo && o < p.hi) w[j >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p.base + o) << (16 * (j & 1));
    } else if (!(j & 1)) {
      if (o >= p.lo && o < p.hi) w[j >> 1] = *reinterpret_cast<const uint32_t*>(p.base + o);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <typename S>
__device__ __forceinline__ S square_sum(const uint4* r, bool bf16) {
  S s = 0;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const uint32_t w[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (bf16) {
        const S a = lo_bf16(w[i]), b = hi_bf16(w[i]);
        s += a * a;
        s += b * b;
      } else {
        const S a = __uint_as_float(w[i]);
        s += a * a;
      }
    }
  }
  return s;
}

// Sum of one double per thread, in thread 0, in a fixed order.  The warps' double
// units are few, so one warp adds for all.
__device__ __forceinline__ double block_sum(double v, double* sh) {
  sh[threadIdx.x] = v;
  __syncthreads();
  double t = 0.0;
  if (threadIdx.x < 32) {
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) t += sh[threadIdx.x + 32 * w];
#pragma unroll
    for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  return t;
}

// partial[cta] (+)= the squares of this launch's chunks cta, cta + grid, ...
template <class Tab>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) grad_square_sum_kernel(const __grid_constant__ Tab t,
                                                                              double* partial, int accumulate) {
  griddep_wait();
  griddep_trigger();
  __shared__ double sh[kThreads];
  double sum = 0.0;
  for (long long c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const Entry& e = t.e[find_entry(t, c)];
    const bool bf16 = e.first & 1;
    const Piece p = piece(e, c);
    uint4 r[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const long long v = p.v0 + j * kThreads;
      r[j] = v < p.nvec ? load_vec<false>(p, v, bf16) : make_uint4(0, 0, 0, 0);
    }
    float s = square_sum<float>(r, bf16);
    if (s > 1.0e-24f && s < 1.0e37f) {
      sum += (double)s;   // no square overflowed; what vanished is below 2^-149 each
    } else {
      uint32_t any = 0;
#pragma unroll
      for (int j = 0; j < kVec; ++j) any |= r[j].x | r[j].y | r[j].z | r[j].w;
      if (any & (bf16 ? 0x7fff7fffu : 0x7fffffffu)) sum += square_sum<double>(r, bf16);
    }
  }
  const double total = block_sum(sum, sh);
  if (threadIdx.x == 0) partial[blockIdx.x] = accumulate ? partial[blockIdx.x] + total : total;
}

// 16 bytes of gradients times f.
__device__ __forceinline__ void scale16(uint32_t* w, float f, bool bf16) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      __nv_bfloat162 b = __floats2bfloat162_rn(lo_bf16(w[i]) * f, hi_bf16(w[i]) * f);
      w[i] = *reinterpret_cast<uint32_t*>(&b);
    } else {
      w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
    }
  }
}

// Every CTA adds the partial sums of all (in the same order), then scales its
// chunks, the list's last ones first.
template <class Tab>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) grad_scale_kernel(const __grid_constant__ Tab t,
                                                                         const double* partial, int partials,
                                                                         float max_norm, float* norm_out,
                                                                         int in_place) {
  griddep_wait();
  griddep_trigger();
  __shared__ double sh[kThreads];
  __shared__ float s_factor;   // negative: no clipping
  __shared__ bool s_tiny;
  double v = 0.0;
  for (int i = threadIdx.x; i < partials; i += kThreads) v += partial[i];
  v = block_sum(v, sh);
  if (threadIdx.x == 0) {
    const double norm = sqrt(v);
    if (blockIdx.x == 0 && norm_out) *norm_out = (float)norm;
    const bool over = norm > (double)max_norm && norm <= 1.7976931348623157e308;   // false for NaN and infinity
    // a factor below fp32's normal range (gradients near its largest value) is taken in two steps
    const double factor = (double)max_norm / norm;
    const bool tiny = factor < 0x1p-126;
    s_factor = over ? (float)(tiny ? factor * 0x1p126 : factor) : -1.f;
    s_tiny = tiny;
  }
  __syncthreads();
  const float f = s_factor;
  const bool clip = f >= 0.f, tiny = s_tiny;
  if (!clip && in_place) return;
  for (long long c = t.chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const Entry& e = t.e[find_entry(t, c)];
    const bool bf16 = e.first & 1;
    const Piece p = piece(e, c);
    char* out = static_cast<char*>(e.out) - p.lo;    // out + o belongs to base + o
    const bool aligned = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    uint4 r[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const long long q = p.v0 + j * kThreads;
      if (q < p.nvec) r[j] = load_vec<true>(p, q, bf16);
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const long long q = p.v0 + j * kThreads;
      if (q >= p.nvec) break;
      uint32_t w[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
      if (clip) {
        scale16(w, f, bf16);
        if (tiny) scale16(w, 0x1p-126f, bf16);   // exact above fp32's normal range
      }
      const long long b = q << 4;
      if (aligned && b >= p.lo && b + 16 <= p.hi) {
        __stcs(reinterpret_cast<uint4*>(out + b), make_uint4(w[0], w[1], w[2], w[3]));
      } else if (bf16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const long long o = b + 2 * i;
          if (o >= p.lo && o < p.hi) *reinterpret_cast<uint16_t*>(out + o) = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const long long o = b + 4 * i;
          if (o >= p.lo && o < p.hi) *reinterpret_cast<uint32_t*>(out + o) = w[i];
        }
      }
    }
  }
}

// The next tensors from t[at] that the table holds, empty ones left out.
template <class Tab>
int fill(Tab& tab, const ClipTensor* t, int n, int at) {
  tab.n = 0;
  tab.chunks = 0;
  for (; at < n && tab.n < Tab::kMax; ++at) {
    if (t[at].numel == 0) continue;
    const long long bytes = t[at].numel * (t[at].bf16 ? 2 : 4) + (long long)(reinterpret_cast<uintptr_t>(t[at].in) & 15);
    Entry& e = tab.e[tab.n++];
    e.in = t[at].in;
    e.out = t[at].out;
    e.numel = t[at].numel;
    e.first = tab.chunks * 2 + (t[at].bf16 ? 1 : 0);
    tab.chunks += ((bytes + 15) / 16 + kChunkVec - 1) / kChunkVec;
  }
  return at;
}

template <class Tab>
cudaError_t run(const ClipTensor* t, int n, float max_norm, float* norm, double* partial, int full, int* launches,
                cudaStream_t s) {
  const bool many = n > Tab::kMax;   // several launches, each adding to the same CTAs' sums
  int in_place = 1;
  for (int i = 0; i < n; ++i)
    if (t[i].numel && t[i].in != t[i].out) in_place = 0;
  Tab tab;
  auto grid_of = [&] { return (int)(tab.chunks < full ? (tab.chunks > 0 ? tab.chunks : 1) : full); };
  int at = 0, partials = 0;
  for (bool first = true; first || at < n; first = false) {
    at = fill(tab, t, n, at);
    partials = many ? full : grid_of();
    cudaError_t e = launch_pdl(grad_square_sum_kernel<Tab>, dim3(partials), dim3(kThreads), 0, s, tab, partial,
                               first ? 0 : 1);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  // the norm alone: no gradient can exceed an infinite limit
  const bool norm_only = in_place && std::isinf(max_norm);
  at = 0;
  for (bool first = true; first || (at < n && !norm_only); first = false) {
    at = many ? fill(tab, t, n, at) : n;   // one table still holds them all
    cudaError_t e = launch_pdl(grad_scale_kernel<Tab>, dim3(norm_only ? 1 : grid_of()), dim3(kThreads), 0, s, tab,
                               static_cast<const double*>(partial), partials, max_norm, first ? norm : nullptr, in_place);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace

int clip_grid(int sms) { return sms * kCtasPerSm; }
size_t clip_workspace_bytes(int sms) { return sizeof(double) * (size_t)clip_grid(sms); }

cudaError_t clip_grad_norm_launch(const ClipTensor* t, int n, float max_norm, float* norm, void* ws, int sms,
                                  int* launches, cudaStream_t s) {
  *launches = 0;
  double* partial = static_cast<double*>(ws);
  return n <= kFewTensors ? run<Table<kFewTensors>>(t, n, max_norm, norm, partial, clip_grid(sms), launches, s)
                          : run<Table<kMaxTensors>>(t, n, max_norm, norm, partial, clip_grid(sms), launches, s);
}

}  // namespace dflash
