// Token embedding with a factor, and its gradient (the drafter's input: an anchor
// token and block_size - 1 mask tokens a block, paper section 4.2):
//
//   out_i = scale E[t_i]            dE[v] (+)= scale sum_{i: t_i = v} d_out_i
//
// The lookup is bound by HBM: rows out, and each distinct row of the table once (8,192 x
// 4,096, bf16 to fp32, 138 MB: 24 us, 5.8 TB/s; 16 rows in 2.5 us).
//
// The gradient.  In a block drafter's training one token, the mask, collects nearly
// all rows, so rows of the table are no unit of work.  One cluster sorts the
// (token, position) pairs by token, positions ascending (a stable radix sort, two
// passes for vocabularies up to 2^18), while the other CTAs zero the gradient (rows with
// a token are written again, which costs less than the sort would by itself).  Then every
// chunk of kEmbedChunk sorted tokens is summed by CTAs of its own: tokens that lie
// inside the chunk go straight to the table's gradient; the sums of a first or last
// token that goes on in another chunk go to memory, and a last kernel adds them in
// order.  No float atomics: the same call gives the same bits.  Sums are fp32, at most
// kEmbedChunk terms, and the chunks' sums are added with their rounding errors carried
// along.  Few tokens take one launch.
//
// What bounds it: HBM where the table is large (8,192 rows of 4,096 into 151,936 bf16:
// 224 us, its 1.38 GB at 6.2 TB/s, of which sort and zeroing 186, sums 29, joins 13), the
// sort and the latency of three launches where it is not (5,470 x 183 into 16,467: 23
// us; 48 x 256, one launch, 5).
#include <algorithm>
#include <type_traits>

#include <cooperative_groups.h>

#include "common.cuh"
#include "embed.cuh"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

constexpr int kChunk = kEmbedChunk;

// ---------------------------------------------------------------- columns of a thread
// A warp takes 32 * W columns.  Where rows allow it (S = 1) a lane has W neighbours, one
// 16-byte access of one type and half or twice that of the other; where they do not (S = 32:
// an odd dim, an odd address) every 32nd, so that the warp's narrow accesses lie side by side
// and a row's bookkeeping still serves W values.  `left`: columns from the lane's first to
// the row's end.
template <int W, int S>
__device__ __forceinline__ int first_column(int unit) {
  return (unit >> 5) * 32 * W + (unit & 31) * (S == 1 ? W : 1);
}
template <typename T, int W>
struct alignas(sizeof(T) * W < 16 ? sizeof(T) * W : 16) Vec {
  T v[W];
};
template <int W, int S, typename T>
__device__ __forceinline__ void load_row(const T* p, int left, float* v) {
  if constexpr (S == 1) {
    const Vec<T, W> x = *reinterpret_cast<const Vec<T, W>*>(p);
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = to_f32<T>(x.v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = j * S < left ? to_f32<T>(p[j * S]) : 0.f;
  }
}
// STREAM: what is written is not read again soon.
template <int W, int S, bool STREAM = false, typename T>
__device__ __forceinline__ void store_row(T* p, int left, const float* v) {
  if constexpr (S == 1) {
    Vec<T, W> x;
#pragma unroll
    for (int j = 0; j < W; ++j) x.v[j] = from_f32<T>(v[j]);
    if constexpr (STREAM && W * sizeof(T) == 16) __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&x));
    else *reinterpret_cast<Vec<T, W>*>(p) = x;
  } else {
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (j * S < left) p[j * S] = from_f32<T>(v[j]);
  }
}
// Values of a lane and their step.
enum Fit { kNarrow, kWide, kWider };   // 16 bytes of neither type, of the wider one, of the narrower one
template <typename A, typename B, int FIT, int NARROW = 4>
struct Columns {
  static constexpr int kMost = sizeof(A) > sizeof(B) ? sizeof(A) : sizeof(B), kLeast = sizeof(A) + sizeof(B) - kMost;
  static constexpr int W = FIT == kNarrow ? NARROW : 16 / (FIT == kWide ? kMost : kLeast), S = FIT == kNarrow ? 32 : 1;
};
// The lookup takes 8 narrow values a lane (20,000 rows of 2,561, bf16 to fp32: 52 us instead
// of 61 with 4), the sums 4 (17,152 x 4,417, fp32, of 29,513 bf16 rows: 229 us, with 8 424).
template <typename A, typename B, int FIT>
using Lookup = Columns<A, B, FIT, 8>;
template <typename A, typename B, int FIT>
bool rows_fit(const void* a, int64_t a_stride, const void* b, int64_t b_stride, int dim) {
  constexpr int W = Columns<A, B, FIT>::W;
  auto fits = [&](const void* p, int64_t stride, int size) {
    const int unit = std::min(16, W * size);
    return reinterpret_cast<uintptr_t>(p) % unit == 0 && stride * size % unit == 0;
  };
  return dim % W == 0 && fits(a, a_stride, sizeof(A)) && fits(b, b_stride, sizeof(B));
}
// run(FIT) of the widest accesses that the rows allow; WIDER: of the narrower type's 16 bytes
template <typename A, typename B, bool WIDER, typename F>
cudaError_t by_fit(const void* a, int64_t a_stride, const void* b, int64_t b_stride, int dim, F run) {
  if constexpr (WIDER && sizeof(A) != sizeof(B)) {
    if (rows_fit<A, B, kWider>(a, a_stride, b, b_stride, dim)) return run(std::integral_constant<int, kWider>{});
  }
  if (rows_fit<A, B, kWide>(a, a_stride, b, b_stride, dim)) return run(std::integral_constant<int, kWide>{});
  return run(std::integral_constant<int, kNarrow>{});
}

// ---------------------------------------------------------------- lookup
// kLookups: accesses of a thread, all loaded before the first is stored.
template <typename TT, typename TO, int FIT, int kLookups>
__global__ void __launch_bounds__(256) embed_kernel(EmbedArgs a) {
  griddep_wait();
  griddep_trigger();
  constexpr int W = Lookup<TT, TO, FIT>::W, S = Lookup<TT, TO, FIT>::S;
  const unsigned units = S == 1 ? a.dim / W : (a.dim + 32 * W - 1) / (32 * W) * 32;   // of a row
  const long long n = (long long)a.n * units, step = (long long)gridDim.x * (256 * kLookups);
  const TT* table = static_cast<const TT*>(a.table);
  TO* out = static_cast<TO*>(a.out);
  for (long long i0 = blockIdx.x * (256LL * kLookups) + threadIdx.x; i0 < n; i0 += step) {
    float v[kLookups][W];
    TO* to[kLookups];
    int left[kLookups];
#pragma unroll
    for (int u = 0; u < kLookups; ++u) {
      const long long i = i0 + u * 256;
      left[u] = 0;
      if (i < n) {
        const int r = n < (1LL << 32) ? (unsigned)i / units : (int)(i / units);
        const int unit = (int)(i - (long long)r * units), c = S == 1 ? unit * W : first_column<W, S>(unit);
        const unsigned t = a.tokens[r];
        to[u] = out + r * a.out_stride + c;
        left[u] = a.dim - c;
        if (t < (unsigned)a.vocab && left[u] > 0) {
          load_row<W, S>(table + (size_t)t * a.dim + c, left[u], v[u]);
        } else {
#pragma unroll
          for (int j = 0; j < W; ++j) v[u][j] = 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kLookups; ++u)
      if (left[u] > 0) {
#pragma unroll
        for (int j = 0; j < W; ++j) v[u][j] *= a.scale;
        store_row<W, S, (kLookups > 1)>(to[u], left[u], v[u]);   // (without: 134 MB of output at 27 us instead of 22.5)
      }
  }
}

// ---------------------------------------------------------------- sort
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9, kBins = 1 << kDigitBits;
constexpr int kMaxCluster = 8;
constexpr int kBatch = 8;   // steps of 32 pairs that a warp loads together
constexpr int kHeld = kSortThreads * kBatch;   // pairs that a CTA can hold
constexpr size_t kSortBytes = sizeof(uint32_t) * kBins * (kSortWarps + kMaxCluster + 1) + sizeof(uint2) * kHeld;

// The lanes that have this lane's digit (kBins: none), by a vote on each bit.
__device__ __forceinline__ unsigned same_digit(unsigned d) {
  unsigned same = 0xffffffffu;
#pragma unroll
  for (int b = 0; b <= kDigitBits; ++b) {
    const bool on = d >> b & 1;
    const unsigned votes = __ballot_sync(0xffffffffu, on);
    same &= on ? votes : ~votes;
  }
  return same;
}

// The share of CTA `cta` of `ctas` in zeroing a table's gradient.
__device__ void zero_fill(void* table, size_t bytes, int cta, int ctas) {
  char* p = static_cast<char*>(table);
  const size_t head = min(bytes, (16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15), vecs = (bytes - head) / 16;
  uint4* v = reinterpret_cast<uint4*>(p + head);
  const size_t step = (size_t)ctas * blockDim.x;
#pragma unroll 4
  for (size_t i = (size_t)cta * blockDim.x + threadIdx.x; i < vecs; i += step) __stcs(v + i, make_uint4(0, 0, 0, 0));
  if (cta == 0) {   // the ends, in the two bytes of the smaller type
    if (threadIdx.x < head / 2) reinterpret_cast<uint16_t*>(p)[threadIdx.x] = 0;
    const size_t tail = head + vecs * 16;
    if (threadIdx.x < (bytes - tail) / 2) reinterpret_cast<uint16_t*>(p + tail)[threadIdx.x] = 0;
  }
}

// The first cluster sorts, the others zero the gradient.  Each warp owns a contiguous
// share of the pairs.  A pass ranks them by digit within the warp, turns the warps'
// counts into places (digits first, then CTAs, then warps, so equal digits keep their
// order) and moves the pairs.  Tokens outside the vocabulary sort behind all others.
// Up to kHeld pairs a CTA stay in registers within a pass and in the cluster's shared
// memory between passes; more go through memory.  (50,001 tokens of 32,003: 27 us, 32 with
// all passes through memory, 39 with digits compared by match.any; 24,026 14.)
__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(EmbedBwdPlan pl, const int32_t* tokens, int passes, void* table,
                                                                     size_t zero_bytes) {
  griddep_wait();
  griddep_trigger();
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), cta = cluster.block_rank();
  if ((int)blockIdx.x >= ctas) {
    zero_fill(table, zero_bytes, blockIdx.x - ctas, gridDim.x - ctas);
    return;
  }
  extern __shared__ __align__(16) uint8_t sort_smem[];
  uint2* held = reinterpret_cast<uint2*>(sort_smem);                 // [kHeld]
  uint32_t* count = reinterpret_cast<uint32_t*>(held + kHeld);       // [warps][bins]
  uint32_t* total = count + kBins * kSortWarps;                      // [CTAs][bins] of every CTA
  uint32_t* place = total + kBins * kMaxCluster;                     // [bins] first place of the CTA's pairs
  __shared__ uint32_t s_scan[kBins / 32], s_valid, s_valids[kMaxCluster];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned below = (1u << lane) - 1;
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");   // all CTAs run before any is written to
  const long long all_warps = (long long)ctas * kSortWarps, me = (long long)cta * kSortWarps + warp;
  const int share = (int)(((pl.n + all_warps - 1) / all_warps + 31) / 32 * 32);   // of a warp
  const int beg = (int)min((long long)pl.n, me * share), end = (int)min((long long)pl.n, (me + 1) * share);
  const bool hold = share <= 32 * kBatch;
  const unsigned of_cta = (unsigned)share * kSortWarps;   // (at most kHeld if held)
  if (tid == 0) s_valid = 0;
  uint2 p[kBatch];
  uint32_t rank[kBatch];
  for (int pass = 0; pass < passes; ++pass) {
    const bool last = pass == passes - 1, last_odd = (passes - pass) & 1;   // the last pass writes `order`
    const uint2* src = last_odd ? pl.spare : pl.order;
    uint2* dst = last_odd ? pl.order : pl.spare;
    const int shift = pass * kDigitBits;
    auto load_batch = [&](int i) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k = i + u * 32 + lane;
        if (k < end) {
          if (pass == 0) p[u] = make_uint2(min((unsigned)tokens[k], (unsigned)pl.vocab), k);
          else p[u] = hold ? held[k - cta * of_cta] : src[k];
        }
      }
    };
    // this batch's ranks among the warp's equal digits; `mine`: what comes before
    uint32_t* mine = count + warp * kBins;
    auto rank_batch = [&](int i) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (i + u * 32 < end) {
          const bool in = i + u * 32 + lane < end;
          const unsigned d = in ? p[u].x >> shift & (kBins - 1) : kBins;
          const unsigned same = same_digit(d);
          const uint32_t before = in ? mine[d] : 0;
          rank[u] = before + __popc(same & below);
          __syncwarp();
          if (in && (same & below) == 0) mine[d] = before + __popc(same);
          __syncwarp();
        }
    };
    load_batch(beg);
    for (int i = tid; i < kBins * kSortWarps; i += kSortThreads) count[i] = 0;
    __syncthreads();
    uint32_t valid = 0;
    for (int i = beg; i < end; i += 32 * kBatch) {
      if (i != beg) load_batch(i);
      rank_batch(i);
      if (pass == 0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) valid += i + u * 32 + lane < end && p[u].x < (unsigned)pl.vocab;
      }
    }
    if (pass == 0) {
      valid = __reduce_add_sync(0xffffffffu, valid);
      if (lane == 0 && valid) atomicAdd(&s_valid, valid);
    }
    __syncthreads();
    if (pass == 0) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (tid < kBins) {
      uint32_t sum = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = count[w * kBins + tid];
        count[w * kBins + tid] = sum;
        sum += c;
      }
      for (int c = 0; c < ctas; ++c) cluster.map_shared_rank(total, c)[cta * kBins + tid] = sum;
    }
    if (pass == 0 && tid == kBins) cluster.map_shared_rank(s_valids, 0)[cta] = s_valid;
    cluster.sync();   // totals are there, and all pairs of the pass in registers (if held)
    if (pass == 0 && cta == 0 && tid == kBins) {
      uint32_t sum = 0;
      for (int c = 0; c < ctas; ++c) sum += s_valids[c];
      *pl.kept = (int)sum;
    }
    uint32_t before = 0, all = 0, run = 0;
    if (tid < kBins) {
      for (int c = 0; c < ctas; ++c) {
        const uint32_t x = total[c * kBins + tid];
        before += c < cta ? x : 0;
        all += x;
      }
      run = all;   // inclusive scan over the digits
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += x;
      }
      if (lane == 31) s_scan[warp] = run;
    }
    __syncthreads();
    if (tid < kBins) {
#pragma unroll
      for (int w = 0; w < kBins / 32; ++w) run += w < warp ? s_scan[w] : 0;
      place[tid] = run - all + before;
    }
    __syncthreads();
    for (int i = beg; i < end; i += 32 * kBatch) {
      if (!hold) {   // again, from the warp's first place on
        load_batch(i);
        rank_batch(i);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (i + u * 32 + lane < end) {
          const unsigned d = p[u].x >> shift & (kBins - 1);
          const unsigned to = place[d] + rank[u] + (hold ? mine[d] : 0);
          if (last || !hold) dst[to] = p[u];
          else cluster.map_shared_rank(held, to / of_cta)[to % of_cta] = p[u];
        }
    }
    // the pairs are where the next pass reads them, and `total` may change (the last
    // pass ends with the kernel)
    if (!last) cluster.sync();
  }
  // no CTA leaves while another may still write its totals or pairs: the last pass' writes
  // to shared memory lie before its cluster.sync
}

// ---------------------------------------------------------------- sums
// A chunk's (or a whole token's) sum into the table's gradient.
template <int W, int S, typename TT>
__device__ __forceinline__ void put_sum(TT* p, int left, const float* sum, float scale, int accumulate) {
  float v[W];
#pragma unroll
  for (int j = 0; j < W; ++j) v[j] = sum[j] * scale;
  if (accumulate) {
    float o[W];
    load_row<W, S>(p, left, o);
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = fmaf(sum[j], scale, o[j]);
  }
  store_row<W, S>(p, left, v);
}

// A chunk's sums over blockDim.x * W columns: a CTA reads each row of d_out in its chunk
// once (50,001 bf16 rows of 1,000 in 35 us, 5.7 TB/s with the rows written).  A token that
// goes on is not followed into the next chunk: longer chains of loads cost what the joins
// save (30,000 rows of 1,001 into 17,152: 72 us instead of 63).
template <typename TO, typename TT, int FIT>
__global__ void __launch_bounds__(256) embed_sum_kernel(EmbedBwdPlan pl, EmbedBwdArgs a) {
  griddep_wait();
  griddep_trigger();
  constexpr int W = Columns<TO, TT, FIT>::W, S = Columns<TO, TT, FIT>::S;
  const int c = first_column<W, S>(blockIdx.y * blockDim.x + threadIdx.x), left = pl.dim - c;
  TT* table = static_cast<TT*>(a.d_table);
  __shared__ uint2 s_pair[kChunk];
  const uint2* order = pl.order;
  const int kept = *pl.kept, i0 = blockIdx.x * kChunk, n = min(kChunk, kept - i0);
  if (n <= 0) return;
  if (threadIdx.x < n) s_pair[threadIdx.x] = order[i0 + threadIdx.x];
  __syncthreads();
  if (c >= pl.dim) return;
  const bool from_before = i0 > 0 && order[i0 - 1].x == s_pair[0].x;
  const bool goes_on = i0 + n < kept && order[i0 + n].x == s_pair[n - 1].x;
  const TO* d_out = static_cast<const TO*>(a.d_out);
  float sum[W] = {};
  bool first = true;
  // loads in flight against CTAs an SM: narrow values 8 rows ahead 229 us, 4 rows 188 (17,152 x
  // 4,417, fp32, of 29,513 bf16 rows); wide ones 16 ahead 96, 8 and 4 73 (32,003 x 1,000 of 50,001)
  constexpr int U = W == 8 || S != 1 ? 4 : 8;
  for (int i = 0; i < n; i += U) {
    float v[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u < n) load_row<W, S>(d_out + (int64_t)s_pair[i + u].y * a.stride + c, left, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = i + u;
      if (k < n) {
#pragma unroll
        for (int j = 0; j < W; ++j) sum[j] += v[u][j];
        const bool last = k == n - 1;
        if (last || s_pair[k + 1].x != s_pair[k].x) {
          const bool head = first && from_before, tail = last && goes_on;
          if (head || tail)   // (a chunk of one token alone has one sum, as its first)
            store_row<W, S>(pl.part + ((size_t)blockIdx.x * 2 + (head ? 0 : 1)) * pl.pitch + c, left, sum);
          else
            put_sum<W, S>(table + (size_t)s_pair[k].x * pl.dim + c, left, sum, a.scale, a.accumulate);
          first = false;
#pragma unroll
          for (int j = 0; j < W; ++j) sum[j] = 0.f;
        }
      }
    }
  }
}

// Tokens that go on from a chunk into others: their chunks' sums in order, with what
// each addition rounds off summed beside them.  A CTA looks at the ends of kJoinChunks
// chunks, over 32 * W columns.  A token of few chunks is one warp's; those of more are
// taken by all warps together, a run of chunks each.
// Latency: order, the search for the token's end, its chunks' sums, the table; 13 us for
// a token of 7,700 rows, 9 for 1,562 chunks of text.  So CTAs an SM count (the whole gradient of
// 50,001 x 1,000 with four columns a lane: three 77.6 us, four 72.5, five 73.7), and warps a CTA
// for long tokens (24,026 x 138, nine tenths one token: 36 us, with four warps 43, sixteen 33; but
// 8,192 x 4,096 225 and, with sixteen, 228).
constexpr int kJoinWarps = 8, kJoinChunks = 8, kJoinAlone = 12;

template <int W>
struct Sum {
  float s[W], e[W];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < W; ++j) s[j] = e[j] = 0.f;
  }
  __device__ __forceinline__ void add(const float* v) {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float t = s[j] + v[j], x = t - s[j];
      e[j] += (s[j] - (t - x)) + (v[j] - x);
      s[j] = t;
    }
  }
  // the sum with its error (which is NaN where the sum is infinite)
  __device__ __forceinline__ void done(float* v) const {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = isfinite(e[j]) ? s[j] + e[j] : s[j];
  }
};

template <typename TT, int W, int S>
__global__ void __launch_bounds__(32 * kJoinWarps, 4) embed_join_kernel(EmbedBwdPlan pl, EmbedBwdArgs a) {
  griddep_wait();
  griddep_trigger();
  __shared__ int s_last[kJoinChunks];              // a chunk's token's last chunk; 0: none begins here and goes on
  __shared__ Sum<W> s_sum[kJoinWarps][32];
  const uint2* order = pl.order;
  const int kept = *pl.kept, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b0 = blockIdx.x * kJoinChunks, c = first_column<W, S>(blockIdx.y * 32 + lane), left = pl.dim - c;
  {
    // lane i: whether the last token of chunk b0 + i begins there and goes on
    const int b = b0 + lane, next = (b + 1) * kChunk;   // a token that goes on reaches the chunk's end
    unsigned t = 0;
    bool goes_on = false;
    if (lane < kJoinChunks && next < kept) {
      t = order[next - 1].x;
      const unsigned after = order[next].x, before = b > 0 ? order[b * kChunk - 1].x : ~0u;
      goes_on = after == t && before != t;
    }
    if (warp == 0 && lane < kJoinChunks) s_last[lane] = 0;
    __syncthreads();
    unsigned todo = __ballot_sync(0xffffffffu, goes_on);
    const int chunks = (kept + kChunk - 1) / kChunk;
    for (int k = 0; todo; ++k, todo &= todo - 1) {
      if (k % kJoinWarps != warp) continue;
      const int i = __ffs(todo) - 1;
      const unsigned token = __shfl_sync(0xffffffffu, t, i);
      // chunk lo begins with the token, chunk hi does not: 32 chunks between them at a time
      int lo = b0 + i + 1, hi = chunks;
      while (hi - lo > 1) {
        const int step = (hi - lo + 32) / 33, at = lo + step * (lane + 1);
        const bool same = at < hi && order[(size_t)at * kChunk].x == token;
        const int n = __popc(__ballot_sync(0xffffffffu, same));
        hi = min(hi, lo + step * (n + 1));
        lo += step * n;
      }
      if (lane == 0) s_last[i] = lo;
    }
  }
  __syncthreads();
  const bool in = c < pl.dim;
  TT* table = static_cast<TT*>(a.d_table) + c;
  // chunks [from, to) of those after b, whose sums are a chunk's first
  auto add_chunks = [&](Sum<W>& sum, int from, int to) {
    constexpr int U = W == 8 ? 4 : 8;
    for (int k = from; k < to; k += U) {
      float v[U][W];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k + u < to) load_row<W, S>(pl.part + (size_t)(k + u) * 2 * pl.pitch + c, left, v[u]);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (k + u < to) sum.add(v[u]);
    }
  };
  auto put = [&](const Sum<W>& sum, int b) {
    float v[W];
    sum.done(v);
    put_sum<W, S>(table + (size_t)order[(b + 1) * kChunk - 1].x * pl.dim, left, v, a.scale, a.accumulate);
  };
  int mine = 0;
  for (int i = 0; i < kJoinChunks; ++i) {
    const int b = b0 + i, last = s_last[i];
    if (!last || last - b > kJoinAlone) continue;
    if (mine++ % kJoinWarps != warp || !in) continue;
    Sum<W> sum;
    sum.zero();
    float v[W];
    load_row<W, S>(pl.part + ((size_t)b * 2 + 1) * pl.pitch + c, left, v);   // b's own: its last token's
    sum.add(v);
    add_chunks(sum, b + 1, last + 1);
    put(sum, b);
  }
  for (int i = 0; i < kJoinChunks; ++i) {
    const int b = b0 + i, last = s_last[i];
    if (!last || last - b <= kJoinAlone) continue;
    const int n = last - b, share = (n + kJoinWarps - 1) / kJoinWarps;
    Sum<W> sum;
    sum.zero();
    if (in) {
      if (warp == 0) {
        float v[W];
        load_row<W, S>(pl.part + ((size_t)b * 2 + 1) * pl.pitch + c, left, v);
        sum.add(v);
      }
      add_chunks(sum, b + 1 + warp * share, min(last + 1, b + 1 + (warp + 1) * share));
    }
    s_sum[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && in) {
      for (int w = 1; w < kJoinWarps; ++w) {
        sum.add(s_sum[w][lane].s);
#pragma unroll
        for (int j = 0; j < W; ++j) sum.e[j] += s_sum[w][lane].e[j];
      }
      put(sum, b);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- few tokens
// One launch: each CTA puts the tokens in order itself (by counting those before each).
// Words of 32 table rows that have a token are taken 32 * W columns at a time: a warp
// sums a token's rows in order, eight warps together those of more than kSmallAlone; the
// other words are zeroed as the bytes that they are.
constexpr int kSmall = 256, kSmallWarps = 8, kSmallAlone = 16;

template <typename TO, typename TT, int FIT>
__global__ void __launch_bounds__(32 * kSmallWarps) embed_small_kernel(EmbedBwdPlan pl, EmbedBwdArgs a) {
  griddep_wait();
  griddep_trigger();
  constexpr int W = Columns<TO, TT, FIT>::W, S = Columns<TO, TT, FIT>::S;
  __shared__ alignas(16) uint64_t s_key[kSmall];
  __shared__ uint32_t s_token[kSmall + 1];
  __shared__ uint16_t s_pos[kSmall], s_first[kSmall];   // s_first: the first token of each word that has one
  __shared__ int s_words;
  __shared__ Sum<W> s_sum[kSmallWarps][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = pl.n;
  static_assert(kSmall == 32 * kSmallWarps, "a token a thread");
  const uint32_t mine = tid < n ? min((unsigned)a.tokens[tid], (unsigned)pl.vocab) : ~0u;
  const uint64_t key = (uint64_t)mine << 32 | tid;
  s_key[tid] = key;
  __syncthreads();
  if (tid < n) {
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 2) {   // (behind the last token: larger than any)
      const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(s_key + j);
      rank += (k.x < key) + (k.y < key);
    }
    s_token[rank] = mine;
    s_pos[rank] = (uint16_t)tid;
  }
  if (tid == 0) s_token[n] = ~0u;
  __syncthreads();
  const int words = (pl.vocab + 31) / 32, tiles = (pl.dim + 32 * W - 1) / (32 * W);
  if (warp == 0) {
    int count = 0;
    for (int i = lane; i < (n + 31) / 32 * 32; i += 32) {
      const bool first = i < n && s_token[i] < (unsigned)pl.vocab && (i == 0 || s_token[i] / 32 != s_token[i - 1] / 32);
      const unsigned votes = __ballot_sync(0xffffffffu, first);
      if (first) s_first[count + __popc(votes & ((1u << lane) - 1))] = (uint16_t)i;
      count += __popc(votes);
    }
    if (lane == 0) s_words = count;
  }
  __syncthreads();
  const int taken = s_words * tiles;
  const TO* d_out = static_cast<const TO*>(a.d_out);
  // the first token that is at least v
  auto find = [&](uint32_t v) {
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_token[mid] >= v) hi = mid; else lo = mid + 1;
    }
    return lo;
  };
  for (int item = blockIdx.x; item < taken + (a.accumulate ? 0 : words); item += gridDim.x) {
    if (item >= taken) {
      const uint32_t v = (item - taken) * 32u;
      const int at = find(v);
      if (at < n && s_token[at] < min(v + 32, (unsigned)pl.vocab)) continue;
      const size_t row = sizeof(TT) * (size_t)pl.dim;
      zero_fill(static_cast<char*>(a.d_table) + v * row, min(32u, pl.vocab - v) * row, 0, 1);
      continue;
    }
    const int w = s_token[s_first[item / tiles]] / 32, c = first_column<W, S>(item % tiles * 32 + lane), left = pl.dim - c;
    const bool in = c < pl.dim;
    TT* table = static_cast<TT*>(a.d_table) + c;
    auto add_rows = [&](Sum<W>& sum, int from, int to) {
      constexpr int U = W == 8 ? 4 : 8;
      for (int k = from; k < to; k += U) {
        float v[U][W];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (k + u < to) load_row<W, S>(d_out + (int64_t)s_pos[k + u] * a.stride + c, left, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (k + u < to) sum.add(v[u]);
      }
    };
    int at = find(w * 32), end_word = find(min(w * 32 + 32, pl.vocab));
    const int rows = min(32, pl.vocab - w * 32);
    if (!a.accumulate) {   // rows without a token
      uint32_t seen = 0;
      for (int k = at; k < end_word; ++k) seen |= 1u << (s_token[k] & 31);
      const float zero[W] = {};
      if (in)
        for (int v = warp; v < rows; v += kSmallWarps)
          if (!(seen >> v & 1)) store_row<W, S>(table + (size_t)(w * 32 + v) * pl.dim, left, zero);
    }
    for (int turn = 0; at < end_word; ++turn) {
      const uint32_t t = s_token[at];
      const int end = find(t + 1);
      float v[W];
      Sum<W> sum;
      sum.zero();
      if (end - at <= kSmallAlone) {
        if (turn % kSmallWarps == warp && in) {
          add_rows(sum, at, end);
          sum.done(v);
          put_sum<W, S>(table + (size_t)t * pl.dim, left, v, a.scale, a.accumulate);
        }
      } else {
        const int share = (end - at + kSmallWarps - 1) / kSmallWarps;
        if (in) add_rows(sum, at + warp * share, min(end, at + (warp + 1) * share));
        s_sum[warp][lane] = sum;
        __syncthreads();
        if (warp == 0 && in) {
          for (int x = 1; x < kSmallWarps; ++x) {
            sum.add(s_sum[x][lane].s);
#pragma unroll
            for (int j = 0; j < W; ++j) sum.e[j] += s_sum[x][lane].e[j];
          }
          sum.done(v);
          put_sum<W, S>(table + (size_t)t * pl.dim, left, v, a.scale, a.accumulate);
        }
        __syncthreads();
      }
      at = end;
    }
  }
}

// ---------------------------------------------------------------- host side
template <typename TT, typename TO, int FIT>
cudaError_t lookup(const EmbedArgs& a, int sms, cudaStream_t s) {
  constexpr int W = Lookup<TT, TO, FIT>::W;
  const long long units = (long long)a.n * (FIT != kNarrow ? a.dim / W : (a.dim + 32 * W - 1) / (32 * W) * 32);
  // few rows: a thread an access, so that the latency is one chain of loads; many: two, which
  // keep more loads in flight (20,000 rows of 2,560, bf16 to fp32: 1, 2, 3, 4 and 8 in 69, 51, 57,
  // 62 and 83 us)
  const bool few = units <= (long long)sms * 2048;
  const long long per = 256 * (few ? 1 : 2);
  const unsigned grid = (unsigned)std::min<long long>((units + per - 1) / per, (long long)sms * 512);
  return few ? launch_pdl(embed_kernel<TT, TO, FIT, 1>, dim3(grid), dim3(256), 0, s, a)
             : launch_pdl(embed_kernel<TT, TO, FIT, 2>, dim3(grid), dim3(256), 0, s, a);
}
template <typename TT, typename TO>
cudaError_t lookup(const EmbedArgs& a, int sms, cudaStream_t s) {
  // 16 bytes of the output a lane, so that a warp's streaming stores are whole lines (20,000 x
  // 2,560, fp32 to bf16: 39 us instead of 45; bf16 to fp32 8,192 x 4,096: two of 16 bytes 26, one 24)
  return by_fit<TT, TO, sizeof(TO) == 2>(a.table, a.dim, a.out, a.out_stride, a.dim,
                                         [&](auto fit) { return lookup<TT, TO, fit()>(a, sms, s); });
}

int passes_of(int vocab) {
  int bits = 0;
  while ((long long)vocab >> bits) ++bits;   // tokens and the one place behind them
  return (bits + kDigitBits - 1) / kDigitBits;
}

cudaError_t sort(const EmbedBwdPlan& pl, const int32_t* tokens, void* table, size_t zero_bytes, int sms, cudaStream_t s) {
  // CTAs that sort: as few as hold the pairs beside a large table (zeroing 1.2 GB takes
  // 186 us beside two, 198 beside eight, which leave SMs without a CTA that zeroes);
  // otherwise as many as have a step a warp to do (5,470 tokens: 17 us with one).
  const int share = zero_bytes > (size_t)64 << 20 ? kHeld : kSortThreads;
  int ctas = 1;
  while (ctas < kMaxCluster && ctas * share < pl.n) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  // CTAs that zero: two an SM, fewer for a small table
  const long long zero = std::min<long long>(2 * sms, (long long)((zero_bytes + 65535) / 65536));
  cfg.gridDim = dim3((unsigned)(ctas + (zero + ctas - 1) / ctas * ctas));
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = kSortBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, embed_sort_kernel, pl, tokens, passes_of(pl.vocab), table, zero_bytes);
}

template <typename TT, int W>
cudaError_t join(const EmbedBwdPlan& pl, const EmbedBwdArgs& a, cudaStream_t s) {
  const dim3 grid((pl.chunks + kJoinChunks - 1) / kJoinChunks, (pl.dim + 32 * W - 1) / (32 * W));
  const bool fits = reinterpret_cast<uintptr_t>(a.d_table) % std::min<size_t>(16, W * sizeof(TT)) == 0 && pl.dim % W == 0;
  return launch_pdl(fits ? embed_join_kernel<TT, W, 1> : embed_join_kernel<TT, W, 32>, grid, dim3(32 * kJoinWarps), 0, s, pl, a);
}
template <typename TO, typename TT, int FIT>
cudaError_t sums(const EmbedBwdPlan& pl, const EmbedBwdArgs& a, int sms, int* launches, cudaStream_t s) {
  constexpr int W = Columns<TO, TT, FIT>::W;
  const int tiles32 = (pl.dim + 32 * W - 1) / (32 * W), words = (pl.vocab + 31) / 32;
  if (pl.n <= kSmall) {
    ++*launches;
    return launch_pdl(embed_small_kernel<TO, TT, FIT>, dim3((unsigned)std::min<long long>((long long)words + (long long)pl.n * tiles32, sms * 2)),
                      dim3(32 * kSmallWarps), 0, s, pl, a);
  }
  cudaError_t e = sort(pl, a.tokens, a.d_table, a.accumulate ? 0 : sizeof(TT) * (size_t)pl.vocab * pl.dim, sms, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  const int threads = std::min(256, tiles32 * 32), tiles = (tiles32 * 32 + threads - 1) / threads;
  e = launch_pdl(embed_sum_kernel<TO, TT, FIT>, dim3(pl.chunks, tiles), dim3(threads), 0, s, pl, a);
  if (e != cudaSuccess) return e;
  *launches += 2;
  // eight columns a lane where there are more CTAs than run at once (30,000 x 1,000: 51 us, with
  // four 54), four where a long token's CTAs work alone (8,192 x 512: 25 us, with eight 29)
  const long long ctas = (long long)((pl.chunks + kJoinChunks - 1) / kJoinChunks) * ((pl.dim + 127) / 128);
  return ctas > 4LL * sms ? join<TT, 8>(pl, a, s) : join<TT, 4>(pl, a, s);
}
template <typename TO, typename TT>
cudaError_t sums(const EmbedBwdPlan& pl, const EmbedBwdArgs& a, int sms, int* launches, cudaStream_t s) {
  // 16 bytes of the table a lane (30,000 x 1,000, fp32 to bf16: 54 us instead of 58; bf16 to fp32
  // 50,001 x 1,000: 72, with 16 bytes of the rows 77)
  return by_fit<TO, TT, sizeof(TT) == 2>(a.d_out, a.stride, a.d_table, pl.dim, pl.dim,
                                         [&](auto fit) { return sums<TO, TT, fit()>(pl, a, sms, launches, s); });
}

}  // namespace

EmbedBwdPlan embed_bwd_plan(void* ws, int n, int dim, int vocab) {
  EmbedBwdPlan pl{};
  pl.n = n;
  pl.vocab = vocab;
  pl.dim = dim;
  pl.pitch = (dim + 7) / 8 * 8;
  pl.chunks = (n + kChunk - 1) / kChunk;
  char* p = static_cast<char*>(ws);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* r = p ? p + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return r;
  };
  pl.kept = reinterpret_cast<int32_t*>(take(256));
  pl.order = reinterpret_cast<uint2*>(take(sizeof(uint2) * (size_t)n));
  pl.spare = reinterpret_cast<uint2*>(take(sizeof(uint2) * (size_t)n));
  pl.part = reinterpret_cast<float*>(take(sizeof(float) * 2 * (size_t)pl.chunks * pl.pitch));
  pl.bytes = off;
  return pl;
}

cudaError_t embed_backward_prepare() {
  return cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSortBytes);
}

cudaError_t embed_launch(const EmbedArgs& a, bool table_f32, bool out_f32, int sms, cudaStream_t s) {
  if (table_f32) return out_f32 ? lookup<float, float>(a, sms, s) : lookup<float, __nv_bfloat16>(a, sms, s);
  return out_f32 ? lookup<__nv_bfloat16, float>(a, sms, s) : lookup<__nv_bfloat16, __nv_bfloat16>(a, sms, s);
}

cudaError_t embed_backward_launch(const EmbedBwdPlan& pl, const EmbedBwdArgs& a, bool out_f32, bool table_f32, int sms,
                                  int* launches, cudaStream_t s) {
  *launches = 0;
  if (out_f32) return table_f32 ? sums<float, float>(pl, a, sms, launches, s) : sums<float, __nv_bfloat16>(pl, a, sms, launches, s);
  return table_f32 ? sums<__nv_bfloat16, float>(pl, a, sms, launches, s)
                   : sums<__nv_bfloat16, __nv_bfloat16>(pl, a, sms, launches, s);
}

}  // namespace dflash
