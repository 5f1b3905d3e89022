// Scoring over the vocabulary: for each row x of logits, z = x / T,
//
//   lse = ln sum_v e^(z_v)          logprob = z_tok - lse
//   H   = lse - sum_v p_v z_v       p_v = e^(z_v - lse)
//   top = the k largest logits, descending, ties to the lowest id
//
// and the gradient of g_lp logprob + g_H H with respect to x,
//
//   dx_v = (1/T) [ g_lp (1[v = tok] - p_v) - g_H p_v (ln p_v + H) ].
//
// Both are bound by HBM: the forward reads every logit once, the gradient
// reads and writes every logit once.  Measured on rows of 151,936 logits: 480 fp32
// rows with 5 alternatives 49.2 us (5.9 TB/s), 2,048 bf16 rows 101 us (6.1 TB/s),
// their gradient 177 us (7.0 TB/s of reads and writes); one fp32 row with 20
// alternatives 9.1 us, which is latency: the launch, 76 KB to each of eight SMs,
// the bar's and the lists' sorts and the cluster's two barriers.
//
// Forward.  A row is one cluster of C CTAs, each taking a C-th of it (C = 1
// where the rows alone fill the GPU, up to 8 for a single row being served),
// so that a call is one launch without scratch memory: the CTAs' statistics
// and candidate lists meet in the first CTA's shared memory.  A thread keeps
// (m, s, t) = (max x, sum e, sum e w) over its logits, w = (x - m) log2(e) / T
// and e = 2^w, rescaled when m grows; the entropy is ln s - ln 2 (t / s), a sum
// of terms of one sign, so nothing cancels.
//
// Top k.  Each warp keeps its k largest (value, id) keys sorted over its
// lanes.  After the first batch of loads, and again after the fourth, the
// sixteenth and so on, the CTA sorts its threads' maxima: the k-th of them, a
// value that k logits are known to reach, is the bar that the rest has to reach
// (hardly more than k of all logits so far do).  A batch whose maximum is below
// the bar costs the top k nothing beyond that maximum, which the softmax needs
// anyway: 600 fp32 rows of 151,936 with 20 alternatives take 61 us (78 with the
// bar set by the first batch alone; a copy's rate allows 54).  Lists are merged in pairs
// (elementwise maximum of one list with the other reversed, then a bitonic
// merge).
#include <cooperative_groups.h>

#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "logprobs.cuh"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values in one register pair: one instruction for both.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
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

// ---------------------------------------------------------------- 16-byte vectors of a row
// A row of V elements whose first lies `mis` elements past a 16-byte boundary
// is covered by aligned vectors 0 .. nvec-1; element u = i * kE + j - mis.
template <typename T> struct Vec {
  static constexpr int kE = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack(uint4 r, float* x, float) {
  x[0] = __uint_as_float(r.x);
  x[1] = __uint_as_float(r.y);
  x[2] = __uint_as_float(r.z);
  x[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(uint4 r, float* x, __nv_bfloat16) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// The largest of a vector's values (NaN aside).
__device__ __forceinline__ float vec_max(uint4 r, float) {
  return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
}
__device__ __forceinline__ float vec_max(uint4 r, __nv_bfloat16) {
  auto as2 = [](uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); };
  const float2 m = __bfloat1622float2(__hmax2(__hmax2(as2(r.x), as2(r.y)), __hmax2(as2(r.z), as2(r.w))));
  return fmaxf(m.x, m.y);
}

// 16 bytes that are read once.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Vector i of the row at `row` (V elements, misalignment mis); elements
// outside the row are -inf and are not read.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, int V, int mis, int i) {
  constexpr int E = Vec<T>::kE;
  const int u0 = i * E - mis;
  if (u0 >= 0 && u0 + E <= V) return load16(row + u0);
  uint32_t w[4];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int u = u0 + j;
      w[j] = u >= 0 && u < V ? reinterpret_cast<const uint32_t*>(row)[u] : 0xff800000u;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int u = u0 + 2 * j + b;
        h[b] = u >= 0 && u < V ? reinterpret_cast<const uint16_t*>(row)[u] : 0xff80u;
      }
      w[j] = h[0] | (h[1] << 16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------- statistics
struct Stats {   // max x, sum e, sum e w with w = (x - m) * scale2, e = 2^w
  float m, s, t;
};

// Statistics about `m` moved to the larger maximum `to`.  The distance is
// clamped where 2^d is 0 anyway, so that a maximum of -inf or of the type's
// lowest value gives 0 and not 0 * inf.  (NaN sums stay NaN.)
__device__ __forceinline__ Stats rescaled(Stats a, float to, float scale2) {
  if (a.m == to) return a;
  const float d = fmaxf((a.m - to) * scale2, -1.0e4f), f = ex2(d);
  return Stats{to, a.s * f, f * (a.t + a.s * d)};
}
__device__ __forceinline__ Stats merged(Stats a, Stats b, float scale2) {
  const float m = fmaxf(a.m, b.m);
  a = rescaled(a, m, scale2);
  b = rescaled(b, m, scale2);
  return Stats{m, a.s + b.s, a.t + b.t};
}
__device__ __forceinline__ Stats warp_merged(Stats v, float scale2) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    v = merged(v, Stats{__shfl_xor_sync(kAll, v.m, o), __shfl_xor_sync(kAll, v.s, o), __shfl_xor_sync(kAll, v.t, o)},
               scale2);
  return v;
}

// ---------------------------------------------------------------- top k
// Orderable key: the larger value first, then the lower id; 0 = no entry
// (no number has it: the id part of a key is never 0).
__device__ __forceinline__ unsigned long long make_key(float x, int id) { return pack_argmax(x + 0.f, id); }   // -0 is 0
__device__ __forceinline__ float key_value(unsigned long long k) {
  const unsigned b = (unsigned)(k >> 32);
  return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}

// Sorted list of a warp: lane i holds the i-th largest key.  A key enters when
// it is larger than thr: the bar, then the list's k-th key once there are k.
struct TopList {
  unsigned long long key, thr;
};
// Whether a batch with maximum m may hold a key above thr: a tie with the bar
// does (its id part is 0), one with a listed key does not (later batches hold
// higher ids).
__device__ __forceinline__ bool reaches(float m, unsigned long long thr) {
  const float x = thr ? key_value(thr) : -INFINITY;
  return static_cast<unsigned>(thr) == 0 ? m >= x : m > x;
}
// Take `key` (the same in every lane) into the list.
__device__ __forceinline__ void insert(TopList& l, unsigned long long key, int k) {
  const int lane = threadIdx.x & 31;
  const int at = __popc(__ballot_sync(kAll, l.key > key));
  const unsigned long long up = __shfl_up_sync(kAll, l.key, 1);
  if (lane == at) l.key = key;
  if (lane > at) l.key = up;
  const unsigned long long kth = __shfl_sync(kAll, l.key, k - 1);
  if (kth > l.thr) l.thr = kth;
}
// Every lane's candidate that beats the threshold.
__device__ __forceinline__ void offer(TopList& l, unsigned long long key, int k) {
  unsigned todo = __ballot_sync(kAll, key > l.thr);
  while (todo) {
    const unsigned long long c = __shfl_sync(kAll, key, __ffs(todo) - 1);
    if (c > l.thr) insert(l, c, k);
    todo &= todo - 1;
  }
}
// The lanes' values in descending order.
__device__ __forceinline__ float sort_desc(float v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int o = k >> 1; o; o >>= 1) {
      const float w = __shfl_xor_sync(kAll, v, o);
      const bool larger = ((lane & o) == 0) == ((lane & k) == 0 || k == 32);   // this lane keeps the larger
      v = larger ? fmaxf(v, w) : fminf(v, w);
    }
  return v;
}
// The 32 largest of two descending lists of values, descending.
__device__ __forceinline__ float merge_values(float a, float b) {
  const int lane = threadIdx.x & 31;
  float v = fmaxf(a, __shfl_sync(kAll, b, 31 - lane));
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float w = __shfl_xor_sync(kAll, v, o);
    v = (lane & o) ? fminf(v, w) : fmaxf(v, w);
  }
  return v;
}
// The 32 largest of two sorted lists, sorted.
__device__ __forceinline__ unsigned long long merge_lists(unsigned long long a, unsigned long long b) {
  const int lane = threadIdx.x & 31;
  const unsigned long long r = __shfl_sync(kAll, b, 31 - lane);
  unsigned long long v = a > r ? a : r;   // bitonic: sort it, the larger to the lower lane
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const unsigned long long w = __shfl_xor_sync(kAll, v, o);
    v = (lane & o) ? (v < w ? v : w) : (v > w ? v : w);
  }
  return v;
}

// ---------------------------------------------------------------- forward
constexpr int kFwdVec = 4;         // vectors a thread loads before it uses any (64 bytes)
constexpr int kMaxCluster = 8;     // the portable cluster size

// grid (C, rows) with clusters of (C, 1, 1): one row a cluster, NT threads a CTA.
template <typename T, bool TOPK, int NT>
__global__ void __launch_bounds__(NT) token_logprobs_kernel(LogprobArgs a, float scale2, float inv_t) {
  griddep_wait();
  griddep_trigger();
  constexpr int E = Vec<T>::kE, kWarps = NT / 32;
  const int C = gridDim.x, part = blockIdx.x, row = blockIdx.y, V = a.vocab, k = a.top_k;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* x = static_cast<const T*>(a.logits) + (size_t)row * a.row_stride;
  const int mis = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const int nvec = (V + mis + E - 1) / E;
  const int i0 = (int)((long long)nvec * part / C), i1 = (int)((long long)nvec * (part + 1) / C);

  cg::cluster_group cluster = cg::this_cluster();
  if (C > 1) cluster.barrier_arrive();   // the first CTA's shared memory is there once every CTA has started

  __shared__ Stats s_stats[kWarps];                                  // the CTA's warps
  __shared__ unsigned long long s_list[TOPK ? kWarps : 1][32];
  __shared__ float s_max[TOPK ? kWarps : 1][32];
  __shared__ Stats c_stats[kMaxCluster];                             // the cluster's CTAs (first CTA's copy)
  __shared__ unsigned long long c_list[TOPK ? kMaxCluster : 1][32];

  // the given token's logit, fetched while the row streams
  int tok = -1;
  float x_tok = 0.f;
  if (part == 0 && tid == 0 && a.tokens) {
    tok = a.tokens[row];
    if (tok >= 0 && tok < V) x_tok = to_f32(x[tok]);
  }

  Stats st{-INFINITY, 0.f, 0.f};
  TopList top{0, 0};
  const uint64_t scale_pair = pack2(scale2, scale2);
  // vectors [full0, full1) of mine lie wholly in the row
  const int full0 = mis ? 1 : 0, full1 = min(i1, (V + mis) / E);
  auto load_batch = [&](int base, uint4* r) {
    if (base >= full0 && base + NT * kFwdVec <= full1) {
      const T* p = x + (ptrdiff_t)(base + tid) * E - mis;
#pragma unroll
      for (int j = 0; j < kFwdVec; ++j) r[j] = load16(p + j * NT * E);
    } else {
#pragma unroll
      for (int j = 0; j < kFwdVec; ++j) {
        const int i = base + tid + j * NT;
        if (i < i1)
          r[j] = load_vec(x, V, mis, i);
        else
          r[j] = sizeof(T) == 4 ? make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u)
                                : make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
      }
    }
  };
  uint4 next[kFwdVec];
  load_batch(i0, next);
  int batch = 0, raise = 0;   // the bar is set by batch 0 and raised by 3, 15, 63, ...
  for (int base = i0; base < i1; base += NT * kFwdVec, ++batch) {
    uint4 r[kFwdVec];
#pragma unroll
    for (int j = 0; j < kFwdVec; ++j) r[j] = next[j];
    if (base + NT * kFwdVec < i1) load_batch(base + NT * kFwdVec, next);   // in flight while this one is used
    float bm = -INFINITY;
#pragma unroll
    for (int j = 0; j < kFwdVec; ++j) bm = fmaxf(bm, vec_max(r[j], T()));
    if (bm > st.m) st = rescaled(st, bm, scale2);
    const float m = st.m == -INFINITY ? 0.f : st.m;   // nothing yet: every e is 0
    const uint64_t minus_m = pack2(-m, -m);
    uint64_t sum = 0, dot = 0;                        // pairs of zeros
#pragma unroll
    for (int j = 0; j < kFwdVec; ++j) {
      float v[E];
      unpack(r[j], v, T());
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 w = unpack2(mul2(add2(pack2(v[e], v[e + 1]), minus_m), scale_pair));
        const uint64_t p = pack2(ex2(w.x), ex2(w.y));
        sum = add2(sum, p);
        dot = fma2(p, pack2(fmaxf(w.x, -1.0e4f), fmaxf(w.y, -1.0e4f)), dot);   // 0 where p is 0, -inf included
      }
    }
    const float2 ds = unpack2(sum), dt = unpack2(dot);
    st.s += ds.x + ds.y;
    st.t += dt.x + dt.y;
    if constexpr (TOPK) {
      if (batch == raise) {   // the bar: the k-th of the threads' maxima so far
        raise = 4 * raise + 3;
        s_max[warp][lane] = sort_desc(st.m);
        __syncthreads();
#pragma unroll
        for (int half = kWarps / 2; half; half >>= 1) {
          if (warp < half) s_max[warp][lane] = merge_values(s_max[warp][lane], s_max[warp + half][lane]);
          __syncthreads();
        }
        const float bar = s_max[0][k - 1];
        __syncthreads();
        // (no bar where fewer than k threads hold a logit above -inf)
        const unsigned long long key = bar == -INFINITY ? 0 : make_key(bar, -1) & 0xffffffff00000000ull;
        if (key > top.thr) top.thr = key;
      }
      if (__any_sync(kAll, reaches(bm, top.thr))) {
#pragma unroll
        for (int j = 0; j < kFwdVec; ++j) {
          if (!__any_sync(kAll, reaches(vec_max(r[j], T()), top.thr))) continue;
          const int i = base + tid + j * NT;
          float v[E];
          unpack(r[j], v, T());
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int u = i * E + e - mis;
            const bool real = i < i1 && u >= 0 && u < V && v[e] == v[e];
            offer(top, real ? make_key(v[e], u) : 0ull, k);
          }
        }
      }
    }
  }

  st = warp_merged(st, scale2);
  if (lane == 0) s_stats[warp] = st;
  if constexpr (TOPK) s_list[warp][lane] = top.key;
  __syncthreads();
  if constexpr (TOPK) {
#pragma unroll
    for (int half = kWarps / 2; half; half >>= 1) {
      if (warp < half) s_list[warp][lane] = merge_lists(s_list[warp][lane], s_list[warp + half][lane]);
      __syncthreads();
    }
  }
  if (warp == 0) {
    st = lane < kWarps ? s_stats[lane] : Stats{-INFINITY, 0.f, 0.f};
    st = warp_merged(st, scale2);
  }
  if (C > 1) {
    cluster.barrier_wait();
    if (warp == 0) {
      if (lane == 0) *cluster.map_shared_rank(&c_stats[part], 0) = st;
      if constexpr (TOPK) *cluster.map_shared_rank(&c_list[part][lane], 0) = s_list[0][lane];
    }
    cluster.sync();
    if (part) return;
    if (warp == 0) {
      st = lane < C ? c_stats[lane] : Stats{-INFINITY, 0.f, 0.f};
      st = warp_merged(st, scale2);
    }
    if constexpr (TOPK) {
      for (int half = C / 2; half; half >>= 1) {   // C is a power of two
        if (warp < half) c_list[warp][lane] = merge_lists(c_list[warp][lane], c_list[warp + half][lane]);
        __syncthreads();
      }
    }
  }
  if (warp) return;
  // a row without a possible token: lse -inf, every log probability -inf, entropy 0
  const bool none = st.m == -INFINITY && st.s == 0.f;
  const float ln_s = logf(st.s);
  if (lane == 0) {
    const float m = st.m == -INFINITY ? 0.f : st.m;
    if (a.lse) a.lse[row] = none ? -INFINITY : m * inv_t + ln_s;
    if (a.entropy) a.entropy[row] = none ? 0.f : ln_s - kLn2 * (st.t / st.s);
    if (a.logprob) {
      float lp = 0.f;   // no token: nothing to score
      if (tok >= 0 && tok < V) lp = none ? -INFINITY : (x_tok - m) * inv_t - ln_s;
      a.logprob[row] = lp;
    }
  }
  if constexpr (TOPK) {
    if (lane < k) {
      const unsigned long long key = C > 1 ? c_list[0][lane] : s_list[0][lane];
      const float m = st.m == -INFINITY ? 0.f : st.m;
      a.top_ids[(size_t)row * k + lane] = key ? unpack_argmax_index(key) : -1;
      a.top_logprobs[(size_t)row * k + lane] =
          none ? -INFINITY : key ? (key_value(key) - m) * inv_t - ln_s : __int_as_float(0x7fc00000);
    }
  }
}

template <typename T, bool TOPK, int NT>
cudaError_t launch_fwd(const LogprobArgs& a, int cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster, a.rows);
  cfg.blockDim = dim3(NT);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, TOPK, NT>, a, logprob_scale2(a.temperature), 1.f / a.temperature);
}

// ---------------------------------------------------------------- gradient
constexpr int kBwdThreads = 256;
constexpr int kBwdVec = 4;

__device__ __forceinline__ void store_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ uint4 repack(const float* v, float) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 repack(const float* v, __nv_bfloat16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct RowGrad {
  float lse, g, gh, a;   // g = g_lp / T, gh = g_H / T, a = -(g + gh H)
  int tok;
  bool zero;
};

// dx of one logit
__device__ __forceinline__ float grad1(float x, int u, const RowGrad& r, float inv_t) {
  const float lp = fmaf(x, inv_t, -r.lse), p = ex2(lp * kLog2e);
  // p (a - gh ln p), 0 where p is 0; NaN logits and sums carry through
  float d = p * fmaf(-r.gh, fmaxf(lp, -1.0e4f), r.a);
  if (u == r.tok) d += r.g;
  return d;
}

// grid (chunks, rows).  Each logit is read before the thread that read it
// writes its gradient, so the two may be the same memory.
template <typename T>
__global__ void __launch_bounds__(kBwdThreads) token_logprobs_backward_kernel(LogprobGradArgs a, float inv_t) {
  griddep_wait();
  griddep_trigger();
  constexpr int E = Vec<T>::kE;
  const int row = blockIdx.y, V = a.vocab;
  const T* x = static_cast<const T*>(a.logits) + (size_t)row * a.row_stride;
  T* d = static_cast<T*>(a.d_logits) + (size_t)row * a.d_row_stride;
  const int mis = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const int mis_d = (int)((reinterpret_cast<uintptr_t>(d) & 15) / sizeof(T));
  const int nvec = (V + mis + E - 1) / E;

  RowGrad r;
  r.lse = a.lse[row];
  r.tok = a.tokens ? a.tokens[row] : -1;
  const bool has = a.d_logprob && r.tok >= 0 && r.tok < V;
  if (!has) r.tok = -1;
  r.g = has ? a.d_logprob[row] * inv_t : 0.f;
  r.gh = a.d_entropy ? a.d_entropy[row] * inv_t : 0.f;
  r.a = -(r.g + (a.d_entropy ? r.gh * a.entropy[row] : 0.f));
  r.zero = r.lse < -1.0e30f;   // nothing but masked logits: no gradient

  const int i_first = blockIdx.x * kBwdThreads * kBwdVec + threadIdx.x;
  if (mis == mis_d) {
    uint4 raw[kBwdVec];
#pragma unroll
    for (int j = 0; j < kBwdVec; ++j) {
      const int i = i_first + j * kBwdThreads;
      if (i < nvec) raw[j] = load_vec(x, V, mis, i);
    }
#pragma unroll
    for (int j = 0; j < kBwdVec; ++j) {
      const int i = i_first + j * kBwdThreads;
      if (i >= nvec) break;
      float v[E];
      unpack(raw[j], v, T());
      const int u0 = i * E - mis;
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = r.zero ? 0.f : grad1(v[e], u0 + e, r, inv_t);
      if (u0 >= 0 && u0 + E <= V) {
        __stcs(reinterpret_cast<uint4*>(d + u0), repack(v, T()));
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (u0 + e >= 0 && u0 + e < V) store_elem(d + u0 + e, v[e]);
      }
    }
  } else {
    // rows whose two alignments differ: element by element, coalesced (2,048 rows of
    // 151,935: 518 us in bf16, 689 in fp32, against 179 and 349 by vectors)
    const int u_first = blockIdx.x * kBwdThreads * kBwdVec * E + threadIdx.x;
#pragma unroll 8
    for (int j = 0; j < kBwdVec * E; ++j) {
      const int u = u_first + j * kBwdThreads;
      if (u < V) store_elem(d + u, r.zero ? 0.f : grad1(to_f32(x[u]), u, r, inv_t));
    }
  }
}

template <typename T>
cudaError_t launch_bwd(const LogprobGradArgs& a, cudaStream_t s) {
  constexpr int E = Vec<T>::kE;
  const int per = kBwdThreads * kBwdVec * E;
  const int chunks = (a.vocab + E - 1 + per - 1) / per;   // up to E - 1 elements of misalignment
  return launch_pdl(token_logprobs_backward_kernel<T>, dim3(chunks, a.rows), dim3(kBwdThreads), 0, s, a,
                    1.f / a.temperature);
}

}  // namespace

cudaError_t token_logprobs_launch(const LogprobArgs& a, bool bf16, int sms, cudaStream_t s) {
  // A row's cluster doubles while that leaves at most 1.25 CTAs an SM and at least two
  // vectors a thread: a row alone is spread over eight SMs (151,936 fp32 logits, 20 alternatives: 27.0 us on
  // one, 11.4 on eight), 77 rows of 32,003 over two each (13.9 on one, 11.7 on two,
  // 12.9 on eight), 1,000 logits stay on one (4.4 us, 7.8 on eight).
  const int nvec = a.vocab / (bf16 ? 8 : 4);
  int cluster = 1;
  while (cluster < kMaxCluster && (long long)a.rows * cluster * 8 <= 5LL * sms && nvec >= 1024 * cluster) cluster *= 2;
  // 512 threads a CTA where there are few CTAs and enough to do for them (one row
  // of 151,936: 9.0 us against 11.4 with 256 threads; 150 rows: 24.7 against 34.5;
  // 600 rows: 68.6 against 61.4).  With bf16 logits they pay only for a handful of
  // rows (one: 9.1 against 11.2, 16: 17.7 against 14.4; 600 rows: 108 against 89, which
  // is slower than fp32's 61 on twice the bytes: with alternatives bf16 takes 79
  // registers, three CTAs an SM, and twice the candidates a load).
  const bool wide = nvec >= 1024 * cluster && (long long)a.rows * cluster <= (bf16 ? sms / 2 : 2 * sms);
  auto launch = [&](auto t, auto topk) {
    using T = decltype(t);
    constexpr bool K = decltype(topk)::value;
    return wide ? launch_fwd<T, K, 512>(a, cluster, s) : launch_fwd<T, K, 256>(a, cluster, s);
  };
  if (bf16) return a.top_k ? launch(__nv_bfloat16(), std::true_type()) : launch(__nv_bfloat16(), std::false_type());
  return a.top_k ? launch(float(), std::true_type()) : launch(float(), std::false_type());
}

cudaError_t token_logprobs_backward_launch(const LogprobGradArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? launch_bwd<__nv_bfloat16>(a, s) : launch_bwd<float>(a, s);
}

}  // namespace dflash
