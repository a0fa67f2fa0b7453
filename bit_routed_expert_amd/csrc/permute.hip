// Rows in expert order and back: the copy of tokens to the rows of their pairs, the weighted sum of
// a token's rows, and the gradients of both. All are bound by the rows' bytes.
#include <algorithm>

#include "internal.h"
#include "elements.h"

namespace moew2 {
namespace {

constexpr int kThreads = 256;

MOEW2_DEV int bin_of(int id, int E) { return (id >= 0 && id < E) ? id : E; }

// Rows beyond the 256 MB that the chip's last cache holds are read and written past it: a reader would find only the
// last ones there, and the passes themselves are faster (805 MB of rows, with and without, its other operands in that cache: the copy 171 and 193 us,
// the weighted sum 162 and 182, the gradient 318 and 347; rows that fit are read up to 15% slower that way).
constexpr long long kCacheBytes = 256LL << 20;

// Pieces of a row of n bytes: piece c lies at byte min(c sizeof(V), n - sizeof(V)), so that the last one overlaps the
// one before it where the row is no whole number of pieces. 16 bytes at any address; less for rows shorter than that.
// (T = 8192, top 8, K = 4097 bf16: 169 us, two bytes at a time 371.)
struct Piece16 { typedef u32x4u_t V; };
struct Piece4 { typedef uint32_t V; };
struct Piece2 { typedef uint16_t V; };
struct Piece1 { typedef uint8_t V; };
template <class P>
MOEW2_DEV typename P::V get(const uint8_t* row, long long c, long long n) {
  return *reinterpret_cast<const typename P::V*>(row + min(c * (long long)sizeof(typename P::V), n - (long long)sizeof(typename P::V)));
}
template <class P, bool PAST>
MOEW2_DEV void put(uint8_t* row, long long c, long long n, const typename P::V& v) {
  auto* p = reinterpret_cast<typename P::V*>(row + min(c * (long long)sizeof(v), n - (long long)sizeof(v)));
  if constexpr (PAST) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// A token's row to the rows of its pairs (row[j], zeros if not here[j]); every `step`th of its pieces from c on.
// `v`: piece c (if there is one).
template <class P, bool PAST>
MOEW2_DEV void copy_row(typename P::V v, long long c, long long step, const uint8_t* __restrict__ x, long long n,
                        uint8_t* __restrict__ rows, int top_k, const int* row, const bool* here) {
  while (c * (long long)sizeof(v) < n) {
    for (int j = 0; j < top_k; ++j) put<P, PAST>(rows + row[j] * n, c, n, here[j] ? v : typename P::V{});
    c += step;
    if (c * (long long)sizeof(v) < n) v = get<P>(x, c, n);
  }
}

// First rows of the bins from their counts: exclusive sums by the whole workgroup, kBinsPer neighbouring bins a
// thread; the caller's count(b) gives bin b's, put(b, first) takes the result.
constexpr int kBinsPer = 1024 / kThreads + 1;
template <class Count, class Put>
MOEW2_DEV void scan_bins(int* wsum /* kThreads / 64 ints of LDS */, Count count, Put put_first) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int v[kBinsPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kBinsPer; ++i) { v[i] = count(tid * kBinsPer + i); sum += v[i]; }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int run = incl - sum;
  for (int w = 0; w < wave; ++w) run += wsum[w];
#pragma unroll
  for (int i = 0; i < kBinsPer; ++i) { put_first(tid * kBinsPer + i, run); run += v[i]; }
}

// Up to kPermuteSmallPairs pairs in one launch: each workgroup finds the rows of its token's pairs by counting
// the pairs that come before them in expert order. Workgroup (T, 0) counts the offsets. That is top_k times as
// many comparisons as pairs, so it loses as their number grows. One launch and three, top 8 of bf16 rows of K =
// 4096: T = 8 4.0 and 8.6 us, 128 7.5 and 10.0, 512 11.4 and 14.9.
constexpr int kMaxTopK = 32;
template <class P, int kPer>
__global__ void __launch_bounds__(kThreads)
permute_small_kernel(int E, int T, int top_k, const int32_t* __restrict__ ids, const uint8_t* __restrict__ x, long long n,
                     uint8_t* __restrict__ rows, int32_t* __restrict__ offsets, int32_t* __restrict__ perm, int32_t* __restrict__ pos) {
  __shared__ int part[kThreads / 64][kMaxTopK];
  __shared__ int key[kMaxTopK];
  __shared__ int row[kMaxTopK];
  __shared__ bool here[kMaxTopK];
  __shared__ int count[kThreads * kBinsPer];
  const int t = blockIdx.x, pairs = T * top_k, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (t == T) {
    if (blockIdx.y) return;
    for (int e = tid; e < kThreads * kBinsPer; e += kThreads) count[e] = 0;
    __syncthreads();
    for (int p = tid; p < pairs; p += kThreads) atomicAdd(&count[bin_of(ids[p], E)], 1);
    __syncthreads();
    scan_bins(part[0], [&](int b) { return count[b]; }, [&](int b, int first) { if (b <= E) offsets[b] = first; });
    return;
  }
  // a pair's key orders pairs by expert, then by index
  auto key_of = [&](int id, int p) { return bin_of(id, E) * kPermuteSmallPairs + p; };
  int k[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) k[i] = ids[min(i * kThreads + tid, pairs - 1)];   // (no branch: the loads go out together)
  const int mine = ids[t * top_k + min(tid, top_k - 1)];
  const long long c = blockIdx.y * kThreads + tid;
  typename P::V v{};
  if (c * (long long)sizeof(v) < n) v = get<P>(x + t * n, c, n);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int q = i * kThreads + tid;
    k[i] = q < pairs ? key_of(k[i], q) : INT32_MAX;
  }
  if (tid < top_k) key[tid] = key_of(mine, t * top_k + tid);
  __syncthreads();
  for (int j = 0; j < top_k; ++j) {
    const int kj = key[j];
    int before = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) before += __popcll(__ballot(k[i] < kj));
    if (lane == 0) part[wave][j] = before;
  }
  __syncthreads();
  if (tid < top_k) {
    const int p = t * top_k + tid;
    int r = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) r += part[w][tid];
    const bool valid = key[tid] / kPermuteSmallPairs < E;
    row[tid] = r;
    here[tid] = valid;
    if (blockIdx.y == 0) {
      perm[r] = p;
      pos[p] = valid ? r : -1 - r;
    }
  }
  __syncthreads();
  copy_row<P, false>(v, c, (long long)gridDim.y * kThreads, x + t * n, n, rows, top_k, row, here);
}

// More pairs, in three launches: ranks and counts of chunks of kChunk pairs, sums of the counts over the chunks
// before, and the copy, whose workgroups add the three parts of a row's index: first row of its expert, pairs of
// the expert in earlier chunks, rank in its chunk. T = 8192, top 8, K = 6144: 162 us
// for 906 MB (5.6 TB/s) with x in the last cache; from memory the copy alone takes 181 - 192, the ranks 10.
constexpr int kChunk = kThreads;

// The lanes of a pair's expert in its wave come from one ballot per bit of the expert; ranks across the waves from
// their counts in LDS.
__global__ void __launch_bounds__(kThreads)
permute_count_kernel(int E, int P, const int32_t* __restrict__ ids, int32_t* __restrict__ rank, int32_t* __restrict__ count) {
  constexpr int kWaves = kThreads / 64;
  __shared__ int hist[kWaves][1024 + 1];
  const int tid = threadIdx.x, wave = tid >> 6, p = blockIdx.x * kChunk + tid;
  const bool inside = p < P;
  const int mine = inside ? bin_of(ids[p], E) : 0;
  for (int e = tid; e <= E; e += kThreads) {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) hist[w][e] = 0;
  }
  uint64_t peers = __ballot(inside);
  for (int b = 0; b < 32 - __clz(E); ++b) {
    const uint64_t set = __ballot(mine >> b & 1);
    peers &= mine >> b & 1 ? set : ~set;
  }
  int r = __popcll(peers & ((1ULL << (tid & 63)) - 1));
  __syncthreads();
  if (inside && r == 0) hist[wave][mine] = __popcll(peers);      // the first of the wave's pairs of its expert
  __syncthreads();
  for (int w = 0; w < wave; ++w) r += hist[w][mine];
  if (inside) rank[p] = r;
  for (int e = tid; e <= E; e += kThreads) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += hist[w][e];
    count[(long long)blockIdx.x * (E + 1) + e] = sum;
  }
}

// count[c][b] becomes the sum over chunks before c; total[b] the sum over all. A workgroup takes kBins bins: a
// group of kThreads / kBins threads each, a run of chunks per thread, kAtOnce of their counts at a time.
constexpr int kBins = 8, kAtOnce = 8;
__global__ void __launch_bounds__(kThreads)
permute_scan_kernel(int bins, int nchunks, int32_t* __restrict__ count, int32_t* __restrict__ total) {
  constexpr int kRuns = kThreads / kBins;
  __shared__ int part[kRuns][kBins];
  const int b = threadIdx.x % kBins, g = threadIdx.x / kBins, bin = blockIdx.x * kBins + b;
  const int per = (nchunks + kRuns - 1) / kRuns, c0 = min(g * per, nchunks), c1 = min(c0 + per, nchunks);
  auto load = [&](int c, int (&v)[kAtOnce]) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) v[i] = count[(long long)min(c + i, nchunks - 1) * bins + min(bin, bins - 1)];
  };
  int sum = 0, v[kAtOnce];
  for (int c = c0; c < c1; c += kAtOnce) {
    load(c, v);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) sum += c + i < c1 ? v[i] : 0;
  }
  part[g][b] = sum;
  __syncthreads();
  int run = 0;
  for (int i = 0; i < g; ++i) run += part[i][b];
  if (bin >= bins) return;
  if (g == kRuns - 1) total[bin] = run + sum;
  for (int c = c0; c < c1; c += kAtOnce) {
    if (per > kAtOnce) load(c, v);                // (else still here)
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (c + i >= c1) break;
      count[(long long)(c + i) * bins + bin] = run;
      run += v[i];
    }
  }
}

// A workgroup takes kThreads / threads tokens, `threads` threads each, so that short rows keep its threads busy
// and tokens share its sums over the experts; kPairs pairs at most.
constexpr int kPairs = kThreads;
template <class P, bool PAST>
__global__ void __launch_bounds__(kThreads)
permute_kernel(int E, int pairs, int top_k, int threads, const int32_t* __restrict__ ids, const int32_t* __restrict__ count,
               const int32_t* __restrict__ total, const int32_t* __restrict__ rank, const uint8_t* __restrict__ x, long long n,
               uint8_t* __restrict__ rows, int32_t* __restrict__ offsets, int32_t* __restrict__ perm, int32_t* __restrict__ pos) {
  __shared__ int first[kThreads * kBinsPer];
  __shared__ int wsum[kThreads / 64];
  __shared__ int row[kPairs];
  __shared__ bool here[kPairs];
  const int tid = threadIdx.x, tokens = kThreads / threads, mine = tid / threads;
  const long long t = (long long)blockIdx.x * tokens + mine, p = (long long)blockIdx.x * tokens * top_k + tid;
  const long long c = (long long)blockIdx.y * threads + tid % threads;
  const bool token = t * top_k < pairs, pair = tid < tokens * top_k && p < pairs;
  typename P::V v{};
  if (token && c * (long long)sizeof(v) < n) v = get<P>(x + t * n, c, n);
  int b = 0, r = 0;
  if (pair) {
    b = bin_of(ids[p], E);
    r = count[p / kChunk * (E + 1) + b] + rank[p];
  }
  scan_bins(wsum, [&](int e) { return e <= E ? total[e] : 0; }, [&](int e, int f) {
    first[e] = f;
    if (e <= E && blockIdx.x == 0 && blockIdx.y == 0) offsets[e] = f;
  });
  __syncthreads();
  if (pair) {
    r += first[b];
    row[tid] = r;
    here[tid] = b < E;
    if (blockIdx.y == 0) {
      perm[r] = (int)p;
      pos[p] = b < E ? r : -1 - r;
    }
  }
  __syncthreads();
  if (token) copy_row<P, PAST>(v, c, (long long)gridDim.y * threads, x + t * n, n, rows, top_k, row + mine * top_k, here + mine * top_k);
}

// y[t] = sum_j w[t, j] rows[pos[t, j]]. W = 8 values a thread, the last 8 of a row where K is no multiple of 8, or 1
// (K < 8). Few tokens: slices of a row to workgroups of their own (blockIdx.y). T = 8192, top 8, K = 6144: 163 us for
// 906 MB (5.6 TB/s); T = 64: 3.4 us. T = 8192, top 8, K = 4097: 123 us, one value a thread 323 (the gradient below
// 253 and 462).
constexpr int kTogether = 8;
template <class T, int W, bool PAST>
__global__ void __launch_bounds__(kThreads)
unpermute_kernel(int top_k, int P, int K, const void* __restrict__ rows, const int32_t* __restrict__ pos,
                 const float* __restrict__ w, void* __restrict__ y) {
  const long long t = blockIdx.x;
  for (int c = threadIdx.x + blockIdx.y * kThreads; c < (K + W - 1) / W; c += kThreads * gridDim.y) {
    const int at = min(W * c, K - W);
    float acc[W];
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < top_k; j0 += kTogether) {      // the loads of some rows together, added in order
      Raw8<T> raw[kTogether];
      float one[kTogether], wt[kTogether];
      bool here[kTogether];
#pragma unroll
      for (int i = 0; i < kTogether; ++i) {
        const int j = j0 + i;
        const int p = j < top_k ? pos[t * top_k + j] : -1;
        here[i] = p >= 0 && p < P;
        if (!here[i]) continue;
        wt[i] = w ? w[t * top_k + j] : 1.f;
        if constexpr (W == 8) raw[i] = load8<T, PAST>(rows, (long long)p * K + at);
        else one[i] = load1<T>(rows, (long long)p * K + at);
      }
#pragma unroll
      for (int i = 0; i < kTogether; ++i) {
        if (!here[i]) continue;
        if constexpr (W == 8) {
          float v[8];
          values8(raw[i], v);
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[q] += wt[i] * v[q];
        } else {
          acc[0] += wt[i] * one[i];
        }
      }
    }
    if constexpr (W == 8) store8<T>(y, t * K + at, raw8<T>(acc));
    else store1<T>(y, t * K + at, acc[0]);
  }
}

// d_rows[pos[t, j]] = w[t, j] dy[t], d_w[t, j] = <dy[t], rows[pos[t, j]]>: TOGETHER rows of a token at a time, so
// that dy is read and the products are summed once for them. The sums are the workgroup's own, in a fixed order.
// d_rows may be rows: then a thread writes no value that another one's product takes, of the last chunk, moved back
// to lie in the row, only those that the chunk before does not hold (T = 8192, K = 510: 42 us over rows, 34
// beside them with the whole chunk written).
// One workgroup per token, four rows together, and one per pair, top 8, bf16: T = 64 with K = 6144 9.2 and 4.1 us,
// 512 19.2 and 17.4, 1024 36.2 and 38.9, 8192 320 (1.7 GB, 5.3 TB/s) and 333; K = 512, T = 8192 31 and 49.
template <class T, int W, int TOGETHER, bool PAST>
__global__ void __launch_bounds__(kThreads)
unpermute_backward_kernel(int top_k, int P, int K, const void* __restrict__ dy, const void* rows,
                          const int32_t* __restrict__ pos, const float* __restrict__ w, void* d_rows,
                          float* __restrict__ d_w) {
  __shared__ float part[kThreads / 64][TOGETHER];
  const long long t = blockIdx.x;
  for (int j0 = blockIdx.y * TOGETHER; j0 < top_k; j0 += gridDim.y * TOGETHER) {
    long long r[TOGETHER];
    float wt[TOGETHER], dot[TOGETHER];
    bool here[TOGETHER], inside[TOGETHER];
#pragma unroll
    for (int i = 0; i < TOGETHER; ++i) {
      const int j = j0 + i, p = j < top_k ? pos[t * top_k + j] : 0;
      r[i] = p >= 0 ? p : -1LL - p;
      inside[i] = j < top_k && r[i] < P;
      here[i] = inside[i] && p >= 0;
      wt[i] = here[i] && w ? w[t * top_k + j] : 1.f;
      dot[i] = 0.f;
    }
    for (int c = threadIdx.x; c < (K + W - 1) / W; c += kThreads) {
      const int at = min(W * c, K - W), again = W * c - at;   // the first `again` values were the last chunk's too
      float d[W];
      if constexpr (W == 8) values8(load8<T>(dy, t * K + at), d);
      else d[0] = load1<T>(dy, t * K + at);
      Raw8<T> raw[TOGETHER];
      float one[TOGETHER];
#pragma unroll
      for (int i = 0; i < TOGETHER; ++i) {
        if (!here[i]) continue;
        if constexpr (W == 8) raw[i] = load8<T, PAST>(rows, r[i] * K + at);
        else one[i] = load1<T>(rows, r[i] * K + at);
      }
#pragma unroll
      for (int i = 0; i < TOGETHER; ++i) {
        if (!inside[i]) continue;
        float o[W];
#pragma unroll
        for (int q = 0; q < W; ++q) o[q] = here[i] ? wt[i] * d[q] : 0.f;
        if constexpr (W == 8) {
          if (again == 0 || d_rows != rows) store8<T, PAST>(d_rows, r[i] * K + at, raw8<T>(o));
          else {
#pragma unroll
            for (int q = 1; q < W; ++q)
              if (q >= again) store1<T>(d_rows, r[i] * K + at + q, o[q]);
          }
        } else {
          store1<T>(d_rows, r[i] * K + at, o[0]);
        }
        if (!here[i]) continue;
        if constexpr (W == 8) {
          float v[8];
          values8(raw[i], v);
#pragma unroll
          for (int q = 0; q < 8; ++q) dot[i] += q < again ? 0.f : d[q] * v[q];
        } else {
          dot[i] += d[0] * one[i];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < TOGETHER; ++i) {
      const float v = wave_sum(dot[i]);
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][i] = v;
    }
    __syncthreads();
    if (threadIdx.x < TOGETHER && j0 + (int)threadIdx.x < top_k) {
      float sum = 0.f;
      for (int i = 0; i < kThreads / 64; ++i) sum += part[i][threadIdx.x];
      d_w[t * top_k + j0 + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

}  // namespace

// ranks, totals, counts of the chunks
size_t permute_workspace_bytes(int E, int P) {
  return align_up((size_t)P * 4) + align_up((size_t)(E + 1) * 4) + align_up((size_t)((P + kChunk - 1) / kChunk) * (E + 1) * 4);
}

// Threads of permute_kernel for a token's row of n pieces (of 16 bytes, as a rule): a wave for short rows, a quarter
// for the shortest. So and with a workgroup each: top 8, T = 65536, n = 8 38 and 106 us; T = 8192, n = 64 22.1 and
// 24.8, n = 256 70 and 58; top 2, T = 65536,
// n = 128 86 and 139.
static int threads_per_token(int top_k, long long n) { return n <= 16 && top_k <= 16 ? 16 : n <= 128 ? 64 : kThreads; }

hipError_t launch_permute(int E, int T, int top_k, const int32_t* ids, const void* x, long long row_bytes, void* rows,
                          int32_t* offsets, int32_t* perm, int32_t* pos, void* workspace, hipStream_t s) {
  const int P = T * top_k, nchunks = (P + kChunk - 1) / kChunk;
  const bool small = P <= kPermuteSmallPairs;
  int32_t *rank = nullptr, *total = nullptr, *count = nullptr;
  if (!small) {
    uint8_t* w = (uint8_t*)workspace;
    rank = (int32_t*)w;   w += align_up((size_t)P * 4);
    total = (int32_t*)w;  w += align_up((size_t)(E + 1) * 4);
    count = (int32_t*)w;
    hipLaunchKernelGGL(permute_count_kernel, dim3(nchunks), dim3(kThreads), 0, s, E, P, ids, rank, count);
    hipLaunchKernelGGL(permute_scan_kernel, dim3((E + kBins) / kBins), dim3(kThreads), 0, s, E + 1, nchunks, count, total);
  }
  auto go = [&](auto piece) {
    typedef decltype(piece) Piece;
    constexpr long long kBytes = sizeof(typename Piece::V);
    const long long n = (row_bytes + kBytes - 1) / kBytes;
    // slices of a row, so that a small batch still has some workgroups per compute unit
    const int slices = (int)std::max<long long>(1, std::min<long long>((n + kThreads - 1) / kThreads, 1024 / (T + 1)));
    if (small) {
      const auto kernel = P <= 2 * kThreads ? permute_small_kernel<Piece, 2> : permute_small_kernel<Piece, kPermuteSmallPairs / kThreads>;
      hipLaunchKernelGGL(kernel, dim3(T + 1, slices), dim3(kThreads), 0, s, E, T, top_k, ids, (const uint8_t*)x, row_bytes,
                         (uint8_t*)rows, offsets, perm, pos);
    } else {
      const auto kernel = (long long)P * row_bytes > kCacheBytes ? permute_kernel<Piece, true> : permute_kernel<Piece, false>;
      const int threads = threads_per_token(top_k, n), tokens = kThreads / threads;
      hipLaunchKernelGGL(kernel, dim3((T + tokens - 1) / tokens, tokens > 1 ? 1 : slices), dim3(kThreads), 0, s, E, P, top_k, threads,
                         ids, count, total, rank, (const uint8_t*)x, row_bytes, (uint8_t*)rows, offsets, perm, pos);
    }
  };
  const uintptr_t bits = (uintptr_t)x | (uintptr_t)rows | (uintptr_t)row_bytes;
  if (row_bytes >= 16) go(Piece16{});
  else if (bits % 4 == 0) go(Piece4{});
  else if (bits % 2 == 0) go(Piece2{});
  else go(Piece1{});
  return hipGetLastError();
}

hipError_t launch_unpermute(int T, int top_k, int K, int dtype, const void* rows, const int32_t* pos, const float* w,
                            void* y, hipStream_t s) {
  with_dtype(dtype, [&](auto t) {
    using TT = decltype(t);
    const bool wide = K >= 8;
    const int n = wide ? (K + 7) / 8 : K, slices = std::max(1, std::min((n + kThreads - 1) / kThreads, 65536 / std::min(T, 65536)));
    const bool past = (long long)T * top_k * K * TT::kBytes > kCacheBytes;
    const auto kernel = !wide ? unpermute_kernel<TT, 1, false> : past ? unpermute_kernel<TT, 8, true> : unpermute_kernel<TT, 8, false>;
    hipLaunchKernelGGL(kernel, dim3(T, slices), dim3(kThreads), 0, s, top_k, T * top_k, K, rows, pos, w, y);
  });
  return hipGetLastError();
}

hipError_t launch_unpermute_backward(int T, int top_k, int K, int dtype, const void* dy, const void* rows,
                                     const int32_t* pos, const float* w, void* d_rows, float* d_w, hipStream_t s) {
  with_dtype(dtype, [&](auto t) {
    using TT = decltype(t);
    const bool wide = K >= 8;
    const bool past = (long long)T * top_k * K * TT::kBytes > kCacheBytes;
    const bool few = T <= 512;
    auto go = [&](auto together) {
      constexpr int N = decltype(together)::value;
      const auto kernel = !wide ? unpermute_backward_kernel<TT, 1, N, false>
                          : past ? unpermute_backward_kernel<TT, 8, N, true> : unpermute_backward_kernel<TT, 8, N, false>;
      hipLaunchKernelGGL(kernel, dim3(T, few ? top_k : 1), dim3(kThreads), 0, s, top_k, T * top_k, K, dy, rows, pos, w, d_rows, d_w);
    };
    if (few || top_k == 1) go(std::integral_constant<int, 1>());
    else if (top_k == 2) go(std::integral_constant<int, 2>());
    else go(std::integral_constant<int, 4>());
  });
  return hipGetLastError();
}

}  // namespace moew2
