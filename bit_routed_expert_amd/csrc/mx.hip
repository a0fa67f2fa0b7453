// MX quantisation and its inverse, and the norm with the residual's addition into MX codes.
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "elements.h"

namespace moew2 {
namespace {

constexpr int kThreads = 256;

// All three kernels are bound by their bytes. Calls whose rows would take more than a quarter of the last cache
// (256 MB) read and write them past it, which leaves it to the codes and their reader and is faster: norm T = 8192
// bf16 with K = 4096 48 -> 41 us, K = 6144 70 -> 61 us (before its codes were exact over the whole range: 43 and 63); 16384 x 4096 values to e2m1 31 -> 28 us
// (with four pieces a thread in flight, which small calls are too small for) and back 34 -> 25 us.
constexpr long long kPastBytes = 64LL << 20;

// Chunks of 8 values; BIG: a call of more than kPastBytes.
template <bool BIG>
constexpr int kPieces = BIG ? 4 : 1;

template <class T, int FMT, bool BIG>
__global__ void __launch_bounds__(kThreads)
mx_quantize_kernel(long long chunks, const void* __restrict__ x, uint8_t* __restrict__ codes,
                   uint8_t* __restrict__ scales) {
  constexpr int N = kPieces<BIG>;
  for (long long c0 = (long long)blockIdx.x * kThreads * N + threadIdx.x; c0 < chunks; c0 += (long long)gridDim.x * kThreads * N) {
    Raw8<T> r[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c0 + i * kThreads < chunks) r[i] = load8<T, BIG>(x, 8 * (c0 + i * kThreads));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (c0 + i * kThreads >= chunks) break;      // (chunks are a multiple of 4: all lanes of a block or none)
      float v[8];
      values8(r[i], v);
      mx_quantize_chunk<FMT>(v, c0 + i * kThreads, codes, scales);
    }
  }
}

template <class T, int FMT, bool BIG>
__global__ void __launch_bounds__(kThreads)
mx_dequantize_kernel(long long chunks, const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                     void* __restrict__ x) {
  for (long long c = (long long)blockIdx.x * kThreads + threadIdx.x; c < chunks; c += (long long)gridDim.x * kThreads) {
    const uint32_t b = scales[c >> 2];
    // 2^(b-127): exponent field b, the subnormal 2^-127 for b = 0, NaN for b = 255
    const float sc = __builtin_bit_cast(float, b == 0 ? 0x00400000u : b == 255u ? 0x7fc00000u : b << 23);
    float v[8];
    if constexpr (FMT == kE2M1) {
      const uint32_t q = *reinterpret_cast<const uint32_t*>(codes + 4 * c);
      static_for<0, 4>([&](auto i) {
        const f32x2e_t f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, decltype(i)::value);
        v[2 * i] = f[0] * sc;
        v[2 * i + 1] = f[1] * sc;
      });
    } else {
      const u32x2_t q = *reinterpret_cast<const u32x2_t*>(codes + 8 * c);
      static_for<0, 8>([&](auto i) {
        v[i] = __builtin_amdgcn_cvt_f32_fp8((int)q[decltype(i)::value / 4], decltype(i)::value % 4) * sc;
      });
    }
    store8<T, BIG>(x, 8 * c, raw8<T>(v));
  }
}

// v rounded to odd, from its rounding to nearest.
MOEW2_DEV float to_odd(double v, float near) {
  const uint32_t b = __builtin_bit_cast(uint32_t, near);
  const double lost = __builtin_fabs(v) - __builtin_fabs((double)near);      // (NaN: no step; an infinity stays one)
  const bool step = (b & 1) == 0 && __builtin_isfinite(near);
  return __builtin_bit_cast(float, b + (step && lost > 0. ? 1u : step && lost < 0. ? ~0u : 0u));
}

// Bound by the rows' bytes while the arithmetic stays below some 40 instructions a value (all of it in double:
// T = 8192, K = 6144 81 us instead of 63). That leaves room for codes of the exact n: sums of squares and 1 / rms in
// double, 1 / rms and the products h gamma as two floats each, of fp32 rows what their fp32 sum leaves out (low). Such
// an n, rounded once to fp32, rounds on to the right element unless it lies on a midpoint of two, whose 19 last bits
// are 0, about once in 2^19 values. The wave computes its values in double from x and residual where one lies there,
// where a sum of two 16-bit values takes more than fp32's 24 bits (they lie 17 binades apart or, in fp16, 14),
// and where the row leaves the range in which none of the products above overflows or loses bits: h 0 or from 2^-40,
// gamma 0 or from 2^-40 to 2^60, 1 / rms from 2^-20 to 2^30, so that h gamma >= 2^-80 and |n| >= 2^-100 are far above 2^-149
// (every chunk computed so: T = 8192, K = 6144 99 us).
// One row per workgroup of NT threads, or, if NT is 64, per wave of a workgroup of four, which needs no barrier:
// the row stays in registers (CH chunks of 8 values a thread). A wave per row and a workgroup per row, bf16 to e4m3:
// T = 8192 with K = 128 5.5 and 8.8 us, 512 8.6 and 10.5, 1024 13.0 and 13.9, 2048 24.4 and 22.8; K = 1024 with T = 1
// 3.6 and 3.0, 1024 4.4 and 4.0, 32768 40 and 53 (all before the codes were made exact, which adds 0.3 to 2.5 us). The
// choice is K's alone, so that the order of a row's sums, and with it every bit of its results, is the same in any
// batch. bf16 to e4m3, T = 1, K = 4096 takes 4.3 us, T = 32 4.9, T = 8192 43 (5.5 TB/s), K = 6144 63 (5.7 TB/s).
template <class T, class G, int FMT, int NT, int CH, bool PAST>
__global__ void __launch_bounds__(NT == 64 ? kThreads : NT)
add_rmsnorm_mx_kernel(int rows, int K, const void* x, const void* residual, const void* __restrict__ gamma, float eps,
                      void* residual_out, void* normed, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr bool kWave = NT == 64;
  const int r = kWave ? (int)blockIdx.x * (kThreads / 64) + ((int)threadIdx.x >> 6) : (int)blockIdx.x;
  if (r >= rows) return;                       // (a whole wave; there is no barrier below then)
  const int tid = kWave ? threadIdx.x & 63 : threadIdx.x;
  const int chunks = K / 8;
  const long long row = (long long)r * chunks;
  constexpr bool kLow = std::is_same<T, F32>::value;
  struct Terms { Raw8<T> x, residual; };                      // (no residual: -0, which, added, changes nothing)
  auto load = [&](int c, Terms& t) {
    t.x = load8<T, PAST>(x, 8 * (row + c));
    if (residual) t.residual = load8<T, PAST>(residual, 8 * (row + c));
    else {
#pragma unroll
      for (auto& v : t.residual.v) v = u32x4_t{} + (T::kBytes == 2 ? 0x80008000u : 0x80000000u);
    }
  };
  float h[CH][8], low[kLow ? CH : 1][8], cross = 0.f;
  bool apart[CH];                                             // a small h, or a sum of two 16-bit values is not exact
  double sum[4] = {0., 0., 0., 0.};
  Terms terms[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i)                                // all loads together
    if (tid + i * NT < chunks) load(tid + i * NT, terms[i]);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * NT;
    if (c >= chunks) continue;
    float v[8];
    values8(terms[i].x, h[i]);
    values8(terms[i].residual, v);
    uint32_t wide = 0, small = ~0u;                           // bits that a sum lost; 2 |h| - 1 of the least h but 0
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (kLow) {
        const double exact = (double)h[i][j] + (double)v[j];
        h[i][j] = (float)exact;
        low[i][j] = (float)(exact - (double)h[i][j]);
        sum[j % 4] = __builtin_fma(exact, exact, sum[j % 4]);
      } else {
        const float both = h[i][j] + v[j], second = both - h[i][j];
        const float lost = (h[i][j] - (both - second)) + (v[j] - second);
        h[i][j] = both;
        wide |= __builtin_bit_cast(uint32_t, lost) << 1;
        cross = __builtin_fmaf(both, lost, cross);
        sum[j % 4] = __builtin_fma((double)both, (double)both, sum[j % 4]);
      }
      small = min(small, (__builtin_bit_cast(uint32_t, h[i][j]) << 1) - 1u);
    }
    apart[i] = wide || small < ((127 - 40) << 24) - 1;
  }
  auto over_row = [&](double v, bool first) {
    v = wave_sum(v);
    if constexpr (!kWave) {
      __shared__ double part[NT / 64];
      if (!first) __syncthreads();
      if ((tid & 63) == 0) part[tid >> 6] = v;
      __syncthreads();
      v = 0.;
#pragma unroll
      for (int w = 0; w < NT / 64; ++w) v += part[w];
    }
    return 1. / __dsqrt_rn(v / (double)K + (double)eps);
  };
  double inv = over_row((sum[0] + sum[1]) + (sum[2] + sum[3]) + 2. * (double)cross, true);
  const bool extreme = !(inv >= 0x1p-20 && inv <= 0x1p30);    // (the whole row's)
  if (!kLow && __builtin_expect(extreme, 0)) {
    double again = 0.;
    for (int c = tid; c < chunks; c += NT) {
      float a[8], v[8];
      Terms t;
      load(c, t);
      values8(t.x, a);
      values8(t.residual, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double exact = (double)a[j] + (double)v[j];
        again = __builtin_fma(exact, exact, again);
      }
    }
    inv = over_row(again, false);
  }
  const float s1 = (float)inv, s2 = (float)(inv - (double)s1);   // inv = s1 + s2
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * NT;
    if (c >= chunks) continue;
    float g[8], n[8], odd[8];
    values8(load8<G>(gamma, 8 * c), g);
    uint32_t least = ~0u;
    float gmin = INFINITY, gmax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      gmin = __builtin_fminf(gmin, __builtin_fabsf(g[j]));
      gmax = __builtin_fmaxf(gmax, __builtin_fabsf(g[j]));
      const float p = h[i][j] * g[j];
      float e = __builtin_fmaf(h[i][j], g[j], -p);
      if constexpr (kLow) e = __builtin_fmaf(low[i][j], g[j], e);
      n[j] = __builtin_copysignf(__builtin_fmaf(p, s1, __builtin_fmaf(p, s2, e * s1)), p);   // (a zero's sign)
      least = min(least, __builtin_bit_cast(uint32_t, n[j]) << 13);
      odd[j] = n[j];
    }
    if (__builtin_expect(__any(gmin < 0x1p-40f), 0)) {        // of those but 0
      gmin = INFINITY;
#pragma unroll
      for (int j = 0; j < 8; ++j) gmin = __builtin_fminf(gmin, g[j] == 0.f ? INFINITY : __builtin_fabsf(g[j]));
    }
    bool alone = extreme || apart[i] || !(gmin >= 0x1p-40f && gmax <= 0x1p60f);
    if (__any(least == 0)) {
      least = 1;
#pragma unroll
      for (int j = 0; j < 8; ++j) least = min(least, n[j] == 0.f ? 1u : __builtin_bit_cast(uint32_t, n[j]) << 13);
      alone |= least == 0;
    }
    if (__builtin_expect(__any(alone), 0)) {
      float a[8], v[8];
      Terms t;
      load(c, t);
      values8(t.x, a);
      values8(t.residual, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double exact = ((double)a[j] + (double)v[j]) * inv * (double)g[j];
        n[j] = (float)exact;
        odd[j] = to_odd(exact, n[j]);
      }
    }
    if (residual_out) store8<T, PAST>(residual_out, 8 * (row + c), raw8<T>(h[i]));
    if (normed) store8<T, PAST>(normed, 8 * (row + c), raw8<T>(n));
    mx_quantize_chunk<FMT>(odd, row + c, codes, scales);
  }
}

inline int grid_of(long long chunks) { return (int)std::min<long long>((chunks + kThreads - 1) / kThreads, 1 << 20); }

}  // namespace

hipError_t launch_mx_quantize(int R, int K, int dtype, const void* x, int format, uint8_t* codes, uint8_t* scales,
                              hipStream_t s) {
  const long long chunks = (long long)R * (K / 8);
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const bool big = 8 * chunks * T::kBytes > kPastBytes;
    const auto kernel = format == kE2M1 ? (big ? mx_quantize_kernel<T, kE2M1, true> : mx_quantize_kernel<T, kE2M1, false>)
                                        : (big ? mx_quantize_kernel<T, kE4M3, true> : mx_quantize_kernel<T, kE4M3, false>);
    const long long threads = big ? (chunks + kPieces<true> - 1) / kPieces<true> : chunks;
    hipLaunchKernelGGL(kernel, dim3(grid_of(threads)), dim3(kThreads), 0, s, chunks, x, codes, scales);
  });
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(int R, int K, int format, const uint8_t* codes, const uint8_t* scales, int dtype,
                                void* x, hipStream_t s) {
  const long long chunks = (long long)R * (K / 8);
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const bool big = 8 * chunks * T::kBytes > kPastBytes;
    const auto kernel = format == kE2M1 ? (big ? mx_dequantize_kernel<T, kE2M1, true> : mx_dequantize_kernel<T, kE2M1, false>)
                                        : (big ? mx_dequantize_kernel<T, kE4M3, true> : mx_dequantize_kernel<T, kE4M3, false>);
    hipLaunchKernelGGL(kernel, dim3(grid_of(chunks)), dim3(kThreads), 0, s, chunks, codes, scales, x);
  });
  return hipGetLastError();
}

hipError_t launch_add_rmsnorm_mx(int T, int K, int dtype, const void* x, const void* residual, const void* gamma,
                                 int gamma_dtype, float eps, void* residual_out, void* normed, int format,
                                 uint8_t* codes, uint8_t* scales, hipStream_t s) {
  with_dtype(dtype, [&](auto t) {
    using TT = decltype(t);
    const bool past = 3LL * T * K * TT::kBytes > kPastBytes;   // x, residual and their sum
    auto go = [&](auto g, auto fmt, auto nt, auto ch) {
      constexpr int NT = decltype(nt)::value, rows = NT == 64 ? kThreads / 64 : 1;
      const auto kernel = past ? add_rmsnorm_mx_kernel<TT, decltype(g), decltype(fmt)::value, NT, decltype(ch)::value, true>
                               : add_rmsnorm_mx_kernel<TT, decltype(g), decltype(fmt)::value, NT, decltype(ch)::value, false>;
      hipLaunchKernelGGL(kernel, dim3((T + rows - 1) / rows), dim3(NT * rows), 0, s, T, K, x, residual, gamma, eps, residual_out, normed,
                         codes, scales);
    };
    typedef std::integral_constant<int, 1> I1;
    typedef std::integral_constant<int, 2> I2;
    typedef std::integral_constant<int, 4> I4;
    typedef std::integral_constant<int, 64> I64;
    typedef std::integral_constant<int, 256> I256;
    typedef std::integral_constant<int, 1024> I1024;
    auto sized = [&](auto g, auto fmt) {
      if (K <= 512) go(g, fmt, I64(), I1());
      else if (K <= 1024) go(g, fmt, I64(), I2());
      else if (K <= 2048) go(g, fmt, I256(), I1());
      else if (K <= 4096) go(g, fmt, I256(), I2());
      else if (K <= kNormWideK) go(g, fmt, I256(), I4());
      else go(g, fmt, I1024(), I4());
    };
    auto formed = [&](auto g) {
      if (format == kE2M1) sized(g, std::integral_constant<int, kE2M1>());
      else sized(g, std::integral_constant<int, kE4M3>());
    };
    if (gamma_dtype == MOE_W2_F32) formed(F32());
    else formed(TT());
  });
  return hipGetLastError();
}

}  // namespace moew2
