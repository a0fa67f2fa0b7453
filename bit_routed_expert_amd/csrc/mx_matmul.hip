// y [M][N] = A [M][K] . W [N][K]^T of MX operands on the block-scaled matrix instruction.
//
// W's rows are the instruction's first operand, A's the second: register r of lane l of a 16 x 16
// accumulator is W row 4 (l / 16) + r, A row l % 16, so a lane holds 4 neighbouring values of one
// row of y. With g = l / 16, instruction s of a step of 512 reduction elements (16 blocks) takes
// block 4s + g as the lane's e2m1 operand (16 code bytes), and, of an e4m3 operand, the 16 values
// 128s + 16g .. and 128s + 64 + 16g ..; the scale it supplies is block 4s + g's in both formats.
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "elements.h"

namespace moew2 {
namespace {

typedef uint32_t u32x2u_t __attribute__((vector_size(8), aligned(1)));    // 8 bytes at any address

// How e4m3 rows of A enter. The instruction adds the products of 8 neighbouring elements in fixed point:
// bits below 2^-13 of the largest product's power of two are dropped (measured with pairs of products; the
// sums of 8, scaled, then add up in fp32). Products with e2m1 never come that low. Of e4m3 elements, whose
// exponents span 15, they do, so those go in as two operands: elements of exponent field 9 .. 15 are multiples
// of 2^-1 below 2^9, those of field 0 .. 8 multiples of 2^-9 below 4, so products with e2m1 (multiples of 1/2,
// largest power 4) keep every bit: 2^-2 = 2^(8 + 2 - 12) and 2^-10 = 2^(1 + 2 - 13). A bf16 result needs that
// too: the elements as they are would leave it off by up to 7 * 2^-13 of the terms' magnitudes where large
// products cancel, and round one in 240 of a product of normal rows (K = 4096) to the other neighbour.
template <int FMT>
MOEW2_DEV f32x4_t mx_mfma_as(const i32x8_t& w, const i32x8_t& a, f32x4_t c, uint32_t sw, uint32_t sa) {
  const f32x4e_t r = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      w, a, __builtin_bit_cast(f32x4e_t, c), kFmtFp4, FMT == kE2M1 ? kFmtFp4 : kFmtFp8, 0, (int)sw, 0, (int)sa);
  return __builtin_bit_cast(f32x4_t, r);
}

MOEW2_DEV void split_e4m3(const i32x8_t& a, i32x8_t& hi, i32x8_t& lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t v = (uint32_t)a[i];
    // bit 7 of each byte whose magnitude bits are at least 0x48 (field 9), spread over the byte
    const uint32_t b = ((v & 0x7f7f7f7fu) + 0x38383838u) & 0x80808080u;
    const uint32_t m = b | (b - (b >> 7));
    hi[i] = (int)(v & m);
    lo[i] = (int)(v & ~m);
  }
}

template <int FMT>
MOEW2_DEV f32x4_t mx_product(const i32x8_t& w, const i32x8_t& a, f32x4_t c, uint32_t sw, uint32_t sa) {
  if constexpr (FMT == kE2M1) return mx_mfma_as<FMT>(w, a, c, sw, sa);
  else {
    i32x8_t hi, lo;
    split_e4m3(a, hi, lo);
    return mx_mfma_as<FMT>(w, lo, mx_mfma_as<FMT>(w, hi, c, sw, sa), sw, sa);
  }
}

// The operands of one row for the four instructions of a step: codes and scales.
template <int FMT>
struct Step {
  u32x4_t codes[4][FMT == kE2M1 ? 1 : 2];
  uint32_t scale[4];   // the lane's scale in byte 0
};

// Step q of a row; `row` is the row's codes, `sc` its scales, nb = K / 32 blocks. LAST: the step may
// reach past the row's end; blocks there are read from the row's last block instead and get code 0
// (e2m1) and scale 1, so they add 0 whatever they hold (an e4m3 operand's own codes stay: 0 of the
// other operand times a value of the same row).
template <int FMT, bool LAST>
MOEW2_DEV void load_step(const uint8_t* row, const uint8_t* sc, int q, int nb, int g, Step<FMT>& st) {
  if constexpr (!LAST) {
    const u32x4u_t s = *reinterpret_cast<const u32x4u_t*>(sc + 16 * q);
#pragma unroll
    for (int i = 0; i < 4; ++i) st.scale[i] = s[i] >> (8 * g);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = 16 * q + 4 * i + g;
    if constexpr (LAST) st.scale[i] = b < nb ? sc[b] : 127u;
    if constexpr (FMT == kE2M1) {
      const int at = LAST ? min(b, nb - 1) : b;
      u32x4_t v = ld16(row + 16 * at);
      if constexpr (LAST) v = b < nb ? v : u32x4_t{0, 0, 0, 0};
      st.codes[i][0] = v;
    } else {
      // halves of blocks: 16-byte piece 2 (16 q + 4 i) + g and the one 4 further
      const int p = 2 * (16 * q + 4 * i) + g;
      st.codes[i][0] = ld16(row + 16 * (LAST ? min(p, 2 * nb - 1) : p));
      st.codes[i][1] = ld16(row + 16 * (LAST ? min(p + 4, 2 * nb - 1) : p + 4));
    }
  }
}

template <int FMT>
MOEW2_DEV i32x8_t operand(const Step<FMT>& st, int i) {
  const u32x4_t& v = st.codes[i][0];
  if constexpr (FMT == kE2M1) return i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
  else {
    const u32x4_t& w = st.codes[i][1];
    return i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], (int)w[0], (int)w[1], (int)w[2], (int)w[3]};
  }
}

// 4 neighbouring values of a row of y (`row`: its first value's index) at column n.
MOEW2_DEV void store4(void* y, long long row, int n, int N, const f32x4_t& v, int out_dtype) {
  if (n + 3 < N) {
    if (out_dtype == MOE_W2_OUT_F32) *reinterpret_cast<u32x4u_t*>((float*)y + row + n) = __builtin_bit_cast(u32x4_t, v);
    else *reinterpret_cast<u32x2u_t*>((char*)y + 2 * (row + n)) = u32x2_t{bf16x2(v[0], v[1]), bf16x2(v[2], v[3])};
    return;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (n + r >= N) break;
    if (out_dtype == MOE_W2_OUT_F32) store1<F32>(y, row + n + r, v[r]);
    else store1<Bf16>(y, row + n + r, v[r]);
  }
}

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// Up to 32 rows of A, bound by the bytes of W: every byte is read once, straight into the operands' registers
// (no other wave needs it, so LDS would only add a wait). One workgroup: 16 rows of W x 16 MT rows of A; the waves
// take the steps in turn, so that N = 4096 keeps 1024 waves loading, and their sums are added in order. N = K =
// 4096, M = 16: 4.4 us for 9 MB with e2m1 rows, 5.4 with e4m3, 4.5 with one such row (an empty kernel takes 2.1).
template <int AFMT, int MT>
__global__ void __launch_bounds__(kThreads)
mx_matmul_rows_kernel(int M, int N, int K, const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_scales,
                      const uint8_t* __restrict__ w_codes, const uint8_t* __restrict__ w_scales, void* __restrict__ y,
                      int out_dtype) {
  __shared__ f32x4_t part[kWaves][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
  const int nb = K / 32;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MT;
  const long long wr = min(n0 + (lane & 15), N - 1);
  const uint8_t* wrow = w_codes + wr * (K / 2);
  const uint8_t* wsc = w_scales + wr * nb;
  const uint8_t* arow[MT];
  const uint8_t* asc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const long long r = min(m0 + 16 * i + (lane & 15), M - 1);
    arow[i] = a_codes + r * (AFMT == kE2M1 ? K / 2 : K);
    asc[i] = a_scales + r * nb;
  }
  f32x4_t acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int full = nb / 16, steps = (nb + 15) / 16;
  auto step = [&](int q, auto last) {
    constexpr bool LAST = decltype(last)::value;
    Step<kE2M1> w;
    load_step<kE2M1, LAST>(wrow, wsc, q, nb, g, w);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      Step<AFMT> a;
      load_step<AFMT, LAST>(arow[i], asc[i], q, nb, g, a);
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i] = mx_product<AFMT>(operand(w, k), operand(a, k), acc[i], w.scale[k], a.scale[k]);
    }
  };
  int q = wave;
  for (; q < full; q += kWaves) step(q, std::false_type());
  if (q < steps) step(q, std::true_type());
#pragma unroll
  for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < MT; i += kWaves) {
    f32x4_t v = part[0][i][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += part[w][i][lane];
    const int m = m0 + 16 * i + (lane & 15), n = n0 + 4 * g;
    if (m >= M) continue;
    store4(y, (long long)m * N, n, N, v, out_dtype);
  }
}


// ------------------------------------------------------------------------------------------
// Larger batches: a workgroup of 4 (or, below, 8) waves computes BM rows of A x BN rows of W, each wave a quarter.
// Stages of BK reduction elements pass through a ring of S buffers in LDS. Codes go there directly
// (buffer_load ... lds); scale bytes, which may lie at any address, through registers. In LDS a row's
// 16-byte chunk c lies in slot c ^ f(row), so that wide reads meet no bank conflict; the direct loads write
// slots in order, so each lane loads the chunk that belongs to its slot. Scale bytes are stored by lane
// group: word g of a row holds block 4 kk + g's byte in byte kk, which instruction kk selects.
// A small tile is bound by the latency of its stages, which the ring covers (M = 128, N = K = 4096: 12.6 us
// with two stages whose loads the compiler waited for early, 7.4 with four), a large one by LDS: at 128 x 128
// the codes that come in and go out take longer than the products.
// ------------------------------------------------------------------------------------------
// A wide LDS read serves 16 lanes at a time, of each 32: 0-3, 12-15, 20-23, 24-27, then the others. f
// spreads the rows and chunks that such lanes ask for (32 rows of one chunk, or 16 rows of two neighbouring
// ones) over the 16 slots of 256 bytes.
template <int CH>   // chunks per row and stage
MOEW2_DEV int slot_of(int row, int c) {
  static_assert(CH == 16 || CH == 8 || CH == 4, "rows of 64, 128 or 256 bytes");
  return c ^ (CH == 4 ? -(row >> 2) & 3 : CH == 8 ? (row >> 1) & 7 : row & 15);
}

// Range of a buffer view of a tile's rows: every offset of theirs is below it (256 rows of at most 2^23
// bytes). The check adds a load's scalar offset without wrapping: a view of 0 bytes reads nothing anywhere.
constexpr uint32_t kViewBytes = 0xfffff000u;

// waits until at most N vector memory operations of this wave are outstanding
template <int N>
MOEW2_DEV void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
// This wave's LDS reads and writes are done, then the workgroup's barrier. The memory clobber keeps every
// access on its side; the waits for the loads in flight are the callers' wait_vm.
MOEW2_DEV void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <int BYTES> struct AnyBytes;              // 1, 2, 4 or 8 bytes at any address
template <> struct AnyBytes<1> { typedef uint8_t type; };
template <> struct AnyBytes<2> { typedef uint16_t type __attribute__((aligned(1))); };
template <> struct AnyBytes<4> { typedef uint32_t type __attribute__((aligned(1))); };
template <> struct AnyBytes<8> { typedef uint64_t type __attribute__((aligned(1))); };

// One operand's share of a stage: ROWS rows of CH chunks and NB scale bytes each. Every wave issues kInstr
// direct loads per stage. Blocks past the row's end get code 0: their loads are out of the buffer's range, so
// they touch no memory and write zeros. EVEN: the rows are whole stages, which saves the masks of the last one
// (M = 8192, N = 4096, 256 x 256 tiles: K = 4064 takes 92 us, K = 4096 85). A branch around loads or products
// would cost more: the compiler moves products, which have no side effect, past branches, and waits for a load
// that it cannot count by waiting for all.
template <int ROWS, int CH, int NB, bool EVEN, int THREADS = kThreads, int SCALERS = THREADS>
struct Operand {
  static constexpr int kCodeBytes = ROWS * CH * 16;
  static constexpr int kScaleBytes = ROWS * NB;
  static constexpr int kInstr = ROWS * CH / THREADS;      // per wave and stage
  static constexpr int kRowsPer = 64 / CH;                // rows per wave instruction
  static constexpr int kPart = ROWS * NB / SCALERS;       // scale bytes per thread and stage (of SCALERS threads)
  static constexpr int kPer = CH / NB;                    // chunks per block
  static_assert(kInstr >= 1 && kPart >= 1 && kPart <= 8, "a stage is a whole number of instructions");
  typedef typename AnyBytes<kPart>::type Part;
  uint32_t off[kInstr];
  const uint8_t* base;                                    // codes and scales of the tile's first row
  const uint8_t* sbase;
  uint32_t soff;                                          // of this thread's row of scales
  int wave, srow_at, sblock;

  MOEW2_DEV void init(const uint8_t* codes, const uint8_t* scales, int first, int rows, int row_bytes, int nb, int w, int lane) {
    wave = w;
    const int last = rows - 1 - first;
    base = codes + (long long)first * row_bytes;
#pragma unroll
    for (int j = 0; j < kInstr; ++j) {
      const int row = (wave * kInstr + j) * kRowsPer + lane / CH;
      off[j] = (uint32_t)min(row, last) * (uint32_t)row_bytes + 16u * slot_of<CH>(row, lane % CH);
    }
    srow_at = (int)(threadIdx.x % SCALERS) * kPart / NB;
    sblock = (int)(threadIdx.x % SCALERS) * kPart % NB;
    sbase = scales + (long long)first * nb;
    soff = (uint32_t)min(srow_at, last) * (uint32_t)nb + (uint32_t)sblock;
  }
  // Loads FROM .. FROM + N - 1 of stage st, of whose blocks `blocks` (0 or less: none) are in the row.
  template <int FROM, int N>
  MOEW2_DEV void load_some(int st, int blocks, uint8_t* codes) const {
    const auto view = buffer_view(base, EVEN && blocks <= 0 ? 0u : kViewBytes);
#pragma unroll
    for (int j = FROM; j < FROM + N; ++j) {
      uint32_t o = off[j];
      if constexpr (!EVEN) {
        const int chunk = slot_of<CH>((wave * kInstr + j) * kRowsPer + (int)(threadIdx.x & 63) / CH, (int)threadIdx.x % CH);
        o |= (uint32_t)((blocks - 1 - chunk / kPer) >> 31);   // all ones past the end
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(view, (__attribute__((address_space(3))) void*)(codes + (wave * kInstr + j) * 1024),
                                               16, (int)o, st * (CH * 16), 0, 0);
    }
  }
  MOEW2_DEV void load(int st, int blocks, uint8_t* codes) const { load_some<0, kInstr>(st, blocks, codes); }
  // This thread's scale bytes of stage st (nb >= kPart): the row's last kPart bytes if it ends before theirs do.
  MOEW2_DEV Part load_scales(int st, int nb) const {
    if constexpr (EVEN) {
      typedef __attribute__((address_space(1))) const uint8_t* global_t;
      global_t p = (global_t)(sbase + min(st * NB, nb - NB));
      asm("" : "+s"(p));   // a scalar base and a 32-bit offset
      return *(__attribute__((address_space(1))) const Part*)(p + soff);
    }
    return *(const Part*)(sbase + (soff + (uint32_t)(min(st * NB, nb - kPart - sblock))));
  }
  // ... with the bytes in their places, 0 (a finite scale of codes 0) past the end
  MOEW2_DEV uint64_t placed(Part v, int st, int nb) const {
    if constexpr (EVEN) return (uint64_t)v;
    const int skip = st * NB + sblock - (nb - kPart);
    return skip <= 0 ? (uint64_t)v : skip >= kPart ? 0 : (uint64_t)v >> (8 * skip);
  }
  MOEW2_DEV void store_scales(uint8_t* scales, uint64_t v) const {
    constexpr int W = NB / 4;                             // bytes per word: instructions per stage
#pragma unroll
    for (int i = 0; i < kPart; ++i) {
      const int blk = sblock + i;
      scales[srow_at * NB + (blk & 3) * W + (blk >> 2)] = (uint8_t)(v >> (8 * i));
    }
  }
};

// 16 rows x 16 F columns of y from one wave's accumulators, turned in LDS (memory of the wave's own, filled
// by the caller, row by row) so that it writes whole pieces of rows. The row stride of 16 F + 4 floats spreads
// the 16 rows of a write over the banks. Rows of y may start anywhere (an odd N): its 16 bytes are stored at any
// address (M = 8200, N = 4100, K = 2080: 110 us element by element, 74 so).
template <int F>
constexpr int kTransposeFloats = 16 * (16 * F + 4);
template <int F>
MOEW2_DEV void store_rows(const float* tp, int lane, void* y, int m0, int n0, int M, int N, int out_dtype) {
  constexpr int stride = 16 * F + 4;
  __builtin_amdgcn_wave_barrier();
  const int rows = min(16, M - m0), cols = min(16 * F, N - n0);
  if (out_dtype == MOE_W2_OUT_BF16) {                      // 8 values, 16 bytes, a lane
    constexpr int per = 2 * F;
#pragma unroll
    for (int q = 0; q < (16 * per + 63) / 64; ++q) {
      const int r = (q * 64 + lane) / per, c = (lane % per) * 8;
      if (r >= rows || c >= cols) continue;             // rows <= 16
      const float* v = tp + r * stride + c;
      const long long o = (long long)(m0 + r) * N + n0 + c;
      if (c + 8 <= cols) {
        const f32x4_t a = *reinterpret_cast<const f32x4_t*>(v), b = *reinterpret_cast<const f32x4_t*>(v + 4);
        *reinterpret_cast<u32x4u_t*>((char*)y + 2 * o) = u32x4_t{bf16x2(a[0], a[1]), bf16x2(a[2], a[3]), bf16x2(b[0], b[1]), bf16x2(b[2], b[3])};
      } else {
#pragma unroll 1
        for (int i = 0; i < cols - c; ++i) store1<Bf16>(y, o + i, v[i]);
      }
    }
  } else {                                                 // 4 values, 16 bytes
    constexpr int per = 4 * F;
#pragma unroll
    for (int q = 0; q < 16 * per / 64; ++q) {
      const int r = (q * 64 + lane) / per, c = (lane % per) * 4;
      if (r >= rows || c >= cols) continue;
      const float* v = tp + r * stride + c;
      const long long o = (long long)(m0 + r) * N + n0 + c;
      if (c + 4 <= cols) {
        *reinterpret_cast<u32x4u_t*>((float*)y + o) = *reinterpret_cast<const u32x4_t*>(v);
      } else {
#pragma unroll 1
        for (int i = 0; i < cols - c; ++i) store1<F32>(y, o + i, v[i]);
      }
    }
  }
  __builtin_amdgcn_wave_barrier();
}

// Tile of this workgroup: workgroups of one XCD (blockIdx % 8) take neighbouring tiles, in columns of 4 row
// tiles, so that they share rows of both operands in the XCD's L2.
MOEW2_DEV void tile_of(int tm, int tn, int& m, int& n) {
  const int total = tm * tn, b = blockIdx.x;
  const int q = total / 8, r = total % 8, x = b % 8;
  const int i = x * q + min(x, r) + b / 8;
  const int per = 4 * tn, group = i / per, rows = min(4, tm - 4 * group), in = i % per;
  m = 4 * group + in % rows;
  n = in / rows;
}

template <int KK> MOEW2_DEV uint32_t scale_word(const uint8_t* p) {
  if constexpr (KK == 1) return *p;
  else if constexpr (KK == 2) return *(const uint16_t*)p;
  else return *(const uint32_t*)p;
}

template <int KKI, int FMT>
MOEW2_DEV f32x4_t mx_mfma_sel(const i32x8_t& w, const i32x8_t& a, f32x4_t c, uint32_t sw, uint32_t sa) {
  const f32x4e_t r = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      w, a, __builtin_bit_cast(f32x4e_t, c), kFmtFp4, FMT == kE2M1 ? kFmtFp4 : kFmtFp8, KKI, (int)sw, KKI, (int)sa);
  return __builtin_bit_cast(f32x4_t, r);
}

template <int AFMT, int BM, int BN, int BK, int S, bool EVEN>
__global__ void __launch_bounds__(kThreads)
mx_matmul_tile_kernel(int M, int N, int K, const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_scales,
                      const uint8_t* __restrict__ w_codes, const uint8_t* __restrict__ w_scales, void* __restrict__ y,
                      int out_dtype) {
  constexpr int CW = BK / 32, CA = AFMT == kE2M1 ? BK / 32 : BK / 16, NB = BK / 32, KK = BK / 128;
  // Waves along M. Four for e4m3 rows of A, whose fragments have twice W's bytes: the same LDS reads as 2 x 2, and
  // each is split by one wave, not two.
  constexpr int WM = AFMT != kE2M1 && BM >= 64 ? 4 : 2, WN = kWaves / WM;
  constexpr int FM = BM / (16 * WM), FN = BN / (16 * WN);   // fragments of 16 rows per wave
  typedef Operand<BN, CW, NB, EVEN> OpW;
  typedef Operand<BM, CA, NB, EVEN> OpA;
  constexpr int kLoads = OpW::kInstr + OpA::kInstr;   // direct loads of a wave per stage
  constexpr int kW = 0, kA = OpW::kCodeBytes, kSW = kA + OpA::kCodeBytes, kSA = kSW + OpW::kScaleBytes,
                kStage = kSA + OpA::kScaleBytes;
  __shared__ __align__(1024) uint8_t lds[S * kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, r16 = lane & 15;
  int tm, tn;
  tile_of((M + BM - 1) / BM, (N + BN - 1) / BN, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int wm = wave % WM * (BM / WM), wn = wave / WM * (BN / WN);
  const int nb = K / 32, stages = (nb + NB - 1) / NB;

  OpW ow;
  OpA oa;
  ow.init(w_codes, w_scales, n0, N, K / 2, nb, wave, lane);
  oa.init(a_codes, a_scales, m0, M, AFMT == kE2M1 ? K / 2 : K, nb, wave, lane);
  typename OpW::Part scw[S];
  typename OpA::Part sca[S];
  auto issue = [&](int st, auto slot) {
    uint8_t* buf = lds + decltype(slot)::value * kStage;
    ow.load(st, nb - NB * st, buf + kW);
    oa.load(st, nb - NB * st, buf + kA);
    scw[decltype(slot)::value] = ow.load_scales(st, nb);
    sca[decltype(slot)::value] = oa.load_scales(st, nb);
  };
  auto store_scales = [&](int st, auto slot) {
    uint8_t* buf = lds + decltype(slot)::value * kStage;
    ow.store_scales(buf + kSW, ow.placed(scw[decltype(slot)::value], st, nb));
    oa.store_scales(buf + kSA, oa.placed(sca[decltype(slot)::value], st, nb));
  };
  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](const uint8_t* buf) {
    uint32_t ws[FN], as[FM];
#pragma unroll
    for (int j = 0; j < FN; ++j) ws[j] = scale_word<KK>(buf + kSW + (wn + 16 * j + r16) * NB + g * KK);
#pragma unroll
    for (int i = 0; i < FM; ++i) as[i] = scale_word<KK>(buf + kSA + (wm + 16 * i + r16) * NB + g * KK);
    static_for<0, KK>([&](auto kkc) {
      constexpr int kk = decltype(kkc)::value;
      i32x8_t w[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int row = wn + 16 * j + r16;
        const u32x4_t v = ld16(buf + kW + (row * CW + slot_of<CW>(r16, 4 * kk + g)) * 16);
        w[j] = i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const uint8_t* row = buf + kA + (wm + 16 * i + r16) * CA * 16;
        if constexpr (AFMT == kE2M1) {
          const u32x4_t v = ld16(row + slot_of<CA>(r16, 4 * kk + g) * 16);
          const i32x8_t a = {(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = mx_mfma_sel<kk, kE2M1>(w[j], a, acc[i][j], ws[j], as[i]);
        } else {
          const u32x4_t v = ld16(row + slot_of<CA>(r16, 8 * kk + g) * 16);
          const u32x4_t u = ld16(row + slot_of<CA>(r16, 8 * kk + g + 4) * 16);
          const i32x8_t a = {(int)v[0], (int)v[1], (int)v[2], (int)v[3], (int)u[0], (int)u[1], (int)u[2], (int)u[3]};
          i32x8_t hi, lo;
          split_e4m3(a, hi, lo);
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = mx_mfma_sel<kk, kE4M3>(w[j], hi, acc[i][j], ws[j], as[i]);
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = mx_mfma_sel<kk, kE4M3>(w[j], lo, acc[i][j], ws[j], as[i]);
        }
      }
    });
  };

  // Loads return in order, so a stage is here once at most the later stages' direct loads are outstanding (their
  // scale loads, which the compiler may place elsewhere, are not counted on).
  static_for<0, S - 1>([&](auto u) { issue(decltype(u)::value, u); });
  wait_vm<(S - 2) * kLoads>();
  store_scales(0, std::integral_constant<int, 0>());
  lds_barrier();
  int st0 = 0;
  for (; st0 + S <= stages; st0 += S) {
    static_for<0, S>([&](auto uc) {
      constexpr int u = decltype(uc)::value;
      typedef std::integral_constant<int, (u + 1) % S> Next;
      issue(st0 + u + S - 1, std::integral_constant<int, (u + S - 1) % S>());
      compute(lds + u * kStage);
      __builtin_amdgcn_sched_barrier(0);   // the products do not sink below the wait for the next loads
      wait_vm<(S - 2) * kLoads>();
      store_scales(st0 + u + 1, Next());
      lds_barrier();
    });
  }
  static_for<0, S - 1>([&](auto uc) {      // what is left of the ring, all of it on its way
    constexpr int u = decltype(uc)::value;
    if (st0 + u >= stages) return;
    compute(lds + u * kStage);
    wait_vm<0>();
    store_scales(st0 + u + 1, std::integral_constant<int, (u + 1) % S>());
    lds_barrier();
  });
  wait_vm<0>();                            // the loads past the end, too, have written their zeros
  lds_barrier();
  static_assert(kWaves * kTransposeFloats<FN> * 4 <= (int)sizeof(lds), "the transposes reuse the ring");
  float* tp = reinterpret_cast<float*>(lds) + wave * kTransposeFloats<FN>;
  static_for<0, FM>([&](auto ic) {
    constexpr int i = decltype(ic)::value;
#pragma unroll
    for (int j = 0; j < FN; ++j) *reinterpret_cast<f32x4_t*>(tp + r16 * (16 * FN + 4) + 16 * j + 4 * g) = acc[i][j];
    store_rows<FN>(tp, lane, y, m0 + wm + 16 * i, n0 + wn, M, N, out_dtype);
  });
}

// ------------------------------------------------------------------------------------------
// Few small tiles, bound by the time that one takes: each wave takes every fourth stage for the whole tile, from a
// ring of its own that no barrier joins, and the four sums are added in order at the end.
// ------------------------------------------------------------------------------------------
template <int AFMT, int BM, int BN, int BK, int S, bool EVEN>
__global__ void __launch_bounds__(kThreads)
mx_matmul_split_kernel(int M, int N, int K, const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_scales,
                       const uint8_t* __restrict__ w_codes, const uint8_t* __restrict__ w_scales, void* __restrict__ y,
                       int out_dtype) {
  constexpr int CW = BK / 32, CA = AFMT == kE2M1 ? BK / 32 : BK / 16, NB = BK / 32, KK = BK / 128;
  constexpr int FM = BM / 16, FN = BN / 16;
  typedef Operand<BN, CW, NB, EVEN, 64> OpW;
  typedef Operand<BM, CA, NB, EVEN, 64> OpA;
  constexpr int kLoads = OpW::kInstr + OpA::kInstr;
  constexpr int kW = 0, kA = OpW::kCodeBytes, kSW = kA + OpA::kCodeBytes, kSA = kSW + OpW::kScaleBytes,
                kStage = kSA + OpA::kScaleBytes;
  typedef std::conditional_t<NB == 8, uint64_t, uint32_t> Row;   // a row's scale bytes of a stage
  typedef std::conditional_t<OpW::kPart == 8, uint64_t, std::conditional_t<OpW::kPart == 4, uint32_t, uint16_t>> PartW;
  typedef std::conditional_t<OpA::kPart == 8, uint64_t, std::conditional_t<OpA::kPart == 4, uint32_t, uint16_t>> PartA;
  static_assert((NB == 4 || NB == 8) && OpW::kPart >= 2 && OpA::kPart >= 2, "scale bytes of a stage in words");
  __shared__ __align__(1024) uint8_t lds[kWaves * S * kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, r16 = lane & 15;
  uint8_t* ring = lds + wave * S * kStage;
  int tm, tn;
  tile_of((M + BM - 1) / BM, (N + BN - 1) / BN, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int nb = K / 32, stages = (nb + NB - 1) / NB, own = (stages + kWaves - 1) / kWaves;   // the last may lie past the end

  OpW ow;
  OpA oa;
  ow.init(w_codes, w_scales, n0, N, K / 2, nb, 0, lane);
  oa.init(a_codes, a_scales, m0, M, AFMT == kE2M1 ? K / 2 : K, nb, 0, lane);
  typename OpW::Part scw[S];
  typename OpA::Part sca[S];
  auto issue = [&](int i, auto slot) {
    const int st = wave + kWaves * i;
    uint8_t* buf = ring + decltype(slot)::value * kStage;
    ow.load(st, nb - NB * st, buf + kW);
    oa.load(st, nb - NB * st, buf + kA);
    scw[decltype(slot)::value] = ow.load_scales(st, nb);
    sca[decltype(slot)::value] = oa.load_scales(st, nb);
  };
  auto store_scales = [&](int i, auto slot) {
    const int st = wave + kWaves * i;
    uint8_t* buf = ring + decltype(slot)::value * kStage;
    const bool here = !EVEN || st < stages;           // past the end: scale 0 with codes 0
    const uint64_t w = here ? ow.placed(scw[decltype(slot)::value], st, nb) : 0;
    const uint64_t a = here ? oa.placed(sca[decltype(slot)::value], st, nb) : 0;
    *reinterpret_cast<PartW*>(buf + kSW + ow.srow_at * NB + ow.sblock) = (PartW)w;
    *reinterpret_cast<PartA*>(buf + kSA + oa.srow_at * NB + oa.sblock) = (PartA)a;
  };
  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](const uint8_t* buf) {
    Row ws[FN], as[FM];
#pragma unroll
    for (int j = 0; j < FN; ++j) ws[j] = *reinterpret_cast<const Row*>(buf + kSW + (16 * j + r16) * NB);
#pragma unroll
    for (int i = 0; i < FM; ++i) as[i] = *reinterpret_cast<const Row*>(buf + kSA + (16 * i + r16) * NB);
    static_for<0, KK>([&](auto kkc) {
      constexpr int kk = decltype(kkc)::value;
      i32x8_t w[FN];
      uint32_t sw[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const u32x4_t v = ld16(buf + kW + ((16 * j + r16) * CW + slot_of<CW>(r16, 4 * kk + g)) * 16);
        w[j] = i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
        sw[j] = (uint32_t)(ws[j] >> (32 * kk)) >> (8 * g);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const uint8_t* row = buf + kA + (16 * i + r16) * CA * 16;
        const uint32_t sa = (uint32_t)(as[i] >> (32 * kk)) >> (8 * g);
        i32x8_t a;
        if constexpr (AFMT == kE2M1) {
          const u32x4_t v = ld16(row + slot_of<CA>(r16, 4 * kk + g) * 16);
          a = i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
        } else {
          const u32x4_t v = ld16(row + slot_of<CA>(r16, 8 * kk + g) * 16);
          const u32x4_t u = ld16(row + slot_of<CA>(r16, 8 * kk + g + 4) * 16);
          a = i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], (int)u[0], (int)u[1], (int)u[2], (int)u[3]};
        }
        if constexpr (AFMT == kE2M1) {
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = mx_mfma_as<AFMT>(w[j], a, acc[i][j], sw[j], sa);
        } else {
          i32x8_t hi, lo;
          split_e4m3(a, hi, lo);
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = mx_mfma_as<AFMT>(w[j], hi, acc[i][j], sw[j], sa);
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = mx_mfma_as<AFMT>(w[j], lo, acc[i][j], sw[j], sa);
        }
      }
    });
  };

  // As in the kernel above, without its barriers: the wave reads only what it loaded. Its reads of a stage have
  // returned (the products took them) before the stage's place is loaded again.
  auto wave_fence = [] { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };
  static_for<0, S - 1>([&](auto u) { issue(decltype(u)::value, u); });
  wait_vm<(S - 2) * kLoads>();
  store_scales(0, std::integral_constant<int, 0>());
  wave_fence();
  int i0 = 0;
  for (; i0 + S <= own; i0 += S) {
    static_for<0, S>([&](auto uc) {
      constexpr int u = decltype(uc)::value;
      typedef std::integral_constant<int, (u + 1) % S> Next;
      issue(i0 + u + S - 1, std::integral_constant<int, (u + S - 1) % S>());
      compute(ring + u * kStage);
      __builtin_amdgcn_sched_barrier(0);
      wait_vm<(S - 2) * kLoads>();
      store_scales(i0 + u + 1, Next());
      wave_fence();
    });
  }
  static_for<0, S - 1>([&](auto uc) {
    constexpr int u = decltype(uc)::value;
    if (i0 + u >= own) return;
    compute(ring + u * kStage);
    wait_vm<0>();
    store_scales(i0 + u + 1, std::integral_constant<int, (u + 1) % S>());
    wave_fence();
  });
  wait_vm<0>();                            // the loads past the end, too, have written their zeros
  lds_barrier();
  // The four sums of a fragment, in order; a wave writes FJ fragments of 16 rows.
  constexpr int FJ = FM * FN / kWaves, kAcross = FN / FJ;
  static_assert(FM * FN % kWaves == 0 && FN % FJ == 0 && FM * kAcross == kWaves, "fragments to a wave");
  static_assert(kWaves * FM * FN * 1024 + kWaves * kTransposeFloats<FJ> * 4 <= (int)sizeof(lds), "the sums reuse the rings");
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) *reinterpret_cast<f32x4_t*>(lds + ((wave * FM + i) * FN + j) * 1024 + lane * 16) = acc[i][j];
  lds_barrier();
  float* tp = reinterpret_cast<float*>(lds + kWaves * FM * FN * 1024) + wave * kTransposeFloats<FJ>;
  const int fi = wave / kAcross, fj = wave % kAcross * FJ;
#pragma unroll
  for (int j = 0; j < FJ; ++j) {
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(lds + (fi * FN + fj + j) * 1024 + lane * 16);
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += *reinterpret_cast<const f32x4_t*>(lds + ((w * FM + fi) * FN + fj + j) * 1024 + lane * 16);
    *reinterpret_cast<f32x4_t*>(tp + r16 * (16 * FJ + 4) + 16 * j + 4 * g) = v;
  }
  store_rows<FJ>(tp, lane, y, m0 + 16 * fi, n0 + 16 * fj, M, N, out_dtype);
}

// ------------------------------------------------------------------------------------------
// The largest products: tiles of 256 x 256, 64 rows of A x 128 of W to each of 8 waves (4 waves of 128 x 128 read
// less LDS, but leave a SIMD one wave, whose every gap shows: M = 8192, N = K = 4096, e4m3 rows to fp32 207 us so,
// 192 with 8; M = N = K = 4096, e2m1 rows 46 and 44). The products are of 32 x 32 x 64 (same rate; the accumulators
// are updated in place, where the compiler kept copying those of 16 x 16 x 128): register r of lane l is W row
// 8 (r / 4) + 4 (l / 32) + r % 4, A row l % 32; with h = l / 32 the lane's e2m1 operand is block h of the 64
// values, its e4m3 operand values 16h .. and 32 + 16h .., its scale block h's.
// A step is 64 reduction elements: 2 groups of a fragment of A with the 4 of W. The reads of a step's
// operands go out in the step before, across stages too: the barrier that hands over a stage sits before
// its last step, when this stage's last reads are done, and the loads of the stage after next follow it.
// M = 8192, N = K = 4096, operands in the last cache: 79 - 85 us with e2m1 rows (3.3 PFLOP/s), 184 - 187 with e4m3;
// from memory 90 - 104 and 204 - 253. e4m3 rows take four times the matrix cycles (half the rate, two operands): 109 us
// of the 184. e2m1 rows are bound by the loads' way to LDS, which only two stages of 64 KB fit: without the products
// 66 us are left, without the operands' reads too 64. Every 4096 more of K takes 72 us, with all rows in the XCD's L2
// 55. (Asking for later stages' rows early, so that they are there, wins 3 to 7% at K = 8192 and loses as much at
// 4096; four stages of half the length take half lines and won nothing.)
// ------------------------------------------------------------------------------------------
typedef float f32x16a_t __attribute__((ext_vector_type(16)));

constexpr int kWideThreads = 512;
template <int AFMT, bool EVEN>
__global__ void __launch_bounds__(kWideThreads)
mx_matmul_wide_kernel(int M, int N, int K, const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_scales,
                      const uint8_t* __restrict__ w_codes, const uint8_t* __restrict__ w_scales, void* __restrict__ y,
                      int out_dtype) {
  constexpr bool four = AFMT == kE2M1;
  constexpr int BM = 256, BN = 256, BK = four ? 256 : 128, FA = 2, FW = 4;
  constexpr int CW = BK / 32, CA = four ? BK / 32 : BK / 16, NB = BK / 32, KS = BK / 64;
  typedef Operand<BN, CW, NB, EVEN, kWideThreads, BN> OpW;
  typedef Operand<BM, CA, NB, EVEN, kWideThreads, BM> OpA;
  typedef OpW Op;   // (its scales: rows and bytes as A's)
  constexpr int kW = 0, kA = OpW::kCodeBytes, kSW = kA + OpA::kCodeBytes, kSA = kSW + OpW::kScaleBytes,
                kStage = kSA + OpA::kScaleBytes;
  __shared__ __align__(1024) uint8_t lds[2 * kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5, r32 = lane & 31;
  int tm, tn;
  tile_of((M + BM - 1) / BM, (N + BN - 1) / BN, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int wm = (wave & 3) * (32 * FA), wn = (wave >> 2) * (32 * FW);
  const int nb = K / 32, stages = (nb + NB - 1) / NB;

  OpW ow;
  OpA oa;
  ow.init(w_codes, w_scales, n0, N, K / 2, nb, wave, lane);
  oa.init(a_codes, a_scales, m0, M, four ? K / 2 : K, nb, wave, lane);

  // Scale bytes: waves 0 - 3 move W's, a row a thread, the others A's. In LDS the bytes of one lane's fragments lie
  // together (KS per fragment), so a lane reads its scales of a stage at once: of F fragments to a wave, row 32 F q +
  // 32 f + r, block 2 ks + h is byte (64 q + 32 h + r) F KS + KS f + ks.
  const bool for_w = wave < BN / 64;
  Op os;
  os.sbase = for_w ? ow.sbase : oa.sbase;
  os.soff = for_w ? ow.soff : oa.soff;
  os.sblock = 0;
  const int srow = threadIdx.x & 255, sf = for_w ? FW : FA;
  const int sat = (for_w ? kSW : kSA) + ((srow / (32 * sf)) * 64 + (srow & 31)) * sf * KS + (srow / 32 % sf) * KS;
  auto store_scales = [&](uint8_t* buf, uint64_t v) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      uint32_t b = 0;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) b |= ((uint32_t)(v >> (8 * (2 * ks + hh))) & 255u) << (8 * ks);
      if constexpr (KS == 2) *reinterpret_cast<uint16_t*>(buf + sat + hh * 32 * sf * KS) = (uint16_t)b;
      else *reinterpret_cast<uint32_t*>(buf + sat + hh * 32 * sf * KS) = b;
    }
  };
  static_assert(OpW::kPart == NB && OpA::kPart == NB && (KS == 2 || KS == 4) && BM == 256 && BN == 256, "one thread per row");

  f32x16a_t acc[FA][FW];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FW; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  u32x4_t w[2][FW], a[2][FA][four ? 1 : 2];      // operands of this step and the next
  constexpr int SW = FW * KS / 4, SA = FA * KS / 4;
  uint32_t sw[SW], sa[SA], nsw[SW], nsa[SA];     // scales of this stage and the next: byte KS f + ks
  typename Op::Part vs;                          // scale bytes of the next stage on their way to LDS

  const int lw = kW + (wn + r32) * CW * 16, la = kA + (wm + r32) * CA * 16;
  auto read = [&](const uint8_t* buf, auto ic, auto parc, auto ksc) {   // fragment i of A, 2 i and 2 i + 1 of W, step ks
    constexpr int i = decltype(ic)::value, par = decltype(parc)::value, ks = decltype(ksc)::value;
#pragma unroll
    for (int f = 2 * i; f < 2 * i + 2; ++f) w[par][f] = ld16(buf + lw + f * CW * 512 + slot_of<CW>(r32, 2 * ks + h) * 16);
    const uint8_t* row = buf + la + i * CA * 512;
    if constexpr (four) a[par][i][0] = ld16(row + slot_of<CA>(r32, 2 * ks + h) * 16);
    else {
      a[par][i][0] = ld16(row + slot_of<CA>(r32, 4 * ks + h) * 16);
      a[par][i][1] = ld16(row + slot_of<CA>(r32, 4 * ks + 2 + h) * 16);
    }
  };
  static_assert(FW == 2 * FA, "two fragments of W are read with one of A");
  auto read_scales = [&](const uint8_t* buf) {
    const uint8_t* pw = buf + kSW + (wn / (32 * FW) * 64 + lane) * FW * KS;
    const uint8_t* pa = buf + kSA + (wm / (32 * FA) * 64 + lane) * FA * KS;
#pragma unroll
    for (int i = 0; i < SW; ++i) nsw[i] = *(const uint32_t*)(pw + 4 * i);
#pragma unroll
    for (int i = 0; i < SA; ++i) nsa[i] = *(const uint32_t*)(pa + 4 * i);
  };
  auto new_scales = [&] {
#pragma unroll
    for (int i = 0; i < SW; ++i) sw[i] = nsw[i];
#pragma unroll
    for (int i = 0; i < SA; ++i) sa[i] = nsa[i];
  };
  auto products = [&](auto ic, auto parc, auto ksc) {   // fragment i of A with the 4 of W
    constexpr int i = decltype(ic)::value, par = decltype(parc)::value, ks = decltype(ksc)::value;
    const u32x4_t& u = a[par][i][0];
    i32x8_t av = {(int)u[0], (int)u[1], (int)u[2], (int)u[3], 0, 0, 0, 0};
    if constexpr (!four) {
#pragma unroll
      for (int q = 0; q < 4; ++q) av[4 + q] = (int)a[par][i][1][q];
    }
    i32x8_t hi = av, lo = av;
    if constexpr (!four) split_e4m3(av, hi, lo);
    static_for<0, FW>([&](auto jc) {
      constexpr int j = decltype(jc)::value, bw = j * KS + ks, ba = i * KS + ks;
      const u32x4_t& v = w[par][j];
      const i32x8_t wv = {(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
      auto mul = [&](const i32x8_t& x) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv, x, acc[i][j], kFmtFp4, four ? kFmtFp4 : kFmtFp8,
                                                                     bw % 4, (int)sw[bw / 4], ba % 4, (int)sa[ba / 4]);
      };
      mul(hi);
      if constexpr (!four) mul(lo);
    });
  };
  // Stage st, in `buf`; `other` holds the next. Stage st + 2 is loaded into `buf` once that is free.
  auto stage = [&](int st, uint8_t* buf, uint8_t* other) {
    static_for<0, KS>([&](auto ksc) {
      constexpr int ks = decltype(ksc)::value, par = ks & 1;
      constexpr bool last = ks == KS - 1;
      typedef std::integral_constant<int, par ^ 1> Next;
      typedef std::integral_constant<int, last ? 0 : ks + 1> NextKs;
      static_for<0, FA>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        if constexpr (ks == KS - 2 && i == FA - 1) {   // the next stage has landed; its scale bytes go to LDS
          wait_vm<0>();
          store_scales(other, os.placed(vs, st + 1, nb));
        }
        if constexpr (last && i == 0) {               // this wave's last reads are done, all waves' next stage is here
          lds_barrier();
          read_scales(other);
        }
        read(last ? other : buf, ic, Next(), NextKs());
        if constexpr (last) {
          constexpr int nw = OpW::kInstr / FA, na = OpA::kInstr / FA;
          ow.template load_some<i * nw, nw>(st + 2, nb - NB * (st + 2), buf + kW);
          oa.template load_some<i * na, na>(st + 2, nb - NB * (st + 2), buf + kA);
          if constexpr (i == FA - 1) vs = os.load_scales(st + 2, nb);
        }
        __builtin_amdgcn_sched_barrier(0);
        products(ic, std::integral_constant<int, par>(), ksc);
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    new_scales();
  };

  uint8_t *buf = lds, *other = lds + kStage;
  typedef std::integral_constant<int, 0> I0;
  ow.load(0, nb, buf + kW);
  oa.load(0, nb, buf + kA);
  vs = os.load_scales(0, nb);
  ow.load(1, nb - NB, other + kW);
  oa.load(1, nb - NB, other + kA);
  store_scales(buf, os.placed(vs, 0, nb));
  vs = os.load_scales(1, nb);
  wait_vm<OpW::kInstr + OpA::kInstr>();
  lds_barrier();
  read_scales(buf);
  new_scales();
  static_for<0, FA>([&](auto i) { read(buf, i, I0(), I0()); });
  for (int st = 0; st < stages; ++st) {
    stage(st, buf, other);
    uint8_t* t = buf;
    buf = other;
    other = t;
  }
  wait_vm<0>();    // the loads past the end, too, have written their zeros
  lds_barrier();
  float* tp = reinterpret_cast<float*>(lds) + wave * kTransposeFloats<2 * FW>;
  static_assert(kWideThreads / 64 * kTransposeFloats<2 * FW> * 4 <= (int)sizeof(lds), "the transposes reuse the stages");
  static_for<0, 2 * FA>([&](auto ic) {   // 16 rows of y at a time: half of a fragment's lanes hold them
    constexpr int i = decltype(ic)::value;
    if ((lane & 16) == 16 * (i & 1)) {
#pragma unroll
      for (int j = 0; j < FW; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<f32x4_t*>(tp + (lane & 15) * (32 * FW + 4) + 32 * j + 8 * q + 4 * h) =
              f32x4_t{acc[i / 2][j][4 * q], acc[i / 2][j][4 * q + 1], acc[i / 2][j][4 * q + 2], acc[i / 2][j][4 * q + 3]};
    }
    store_rows<2 * FW>(tp, lane, y, m0 + wm + 16 * i, n0 + wn, M, N, out_dtype);
  });
}

}  // namespace

hipError_t launch_mx_matmul(int M, int N, int K, int a_format, const uint8_t* a_codes, const uint8_t* a_scales,
                            const uint8_t* w_codes, const uint8_t* w_scales, void* y, int out_dtype, hipStream_t s) {
  auto go = [&](auto afmt, auto mt) {
    constexpr int MT = decltype(mt)::value;
    // grid rows are 16 bits: larger batches go in slices of rows
    const int slice = 65535 * 16 * MT;
    for (long long m = 0; m < M; m += slice) {
      const int rows = (int)std::min<long long>(slice, M - m);
      constexpr int AF = decltype(afmt)::value;
      hipLaunchKernelGGL((mx_matmul_rows_kernel<AF, MT>), dim3((N + 15) / 16, (rows + 16 * MT - 1) / (16 * MT)), dim3(kThreads), 0, s,
                         rows, N, K, a_codes + m * (AF == kE2M1 ? K / 2 : K), a_scales + m * (K / 32), w_codes, w_scales,
                         (char*)y + m * N * (out_dtype == MOE_W2_OUT_F32 ? 4 : 2), out_dtype);
    }
  };
  auto split = [&](auto afmt, auto bm, auto bn, auto ring) {
    constexpr int AF = decltype(afmt)::value, BM = decltype(bm)::value, BN = decltype(bn)::value, S = decltype(ring)::value;
    const auto kernel = K % 256 ? mx_matmul_split_kernel<AF, BM, BN, 256, S, false> : mx_matmul_split_kernel<AF, BM, BN, 256, S, true>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((long long)((M + BM - 1) / BM) * ((N + BN - 1) / BN))), dim3(kThreads), 0, s,
                       M, N, K, a_codes, a_scales, w_codes, w_scales, y, out_dtype);
  };
  auto tiles = [&](auto afmt, auto bm, auto bn, auto bk, auto ring) {
    constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value;
    constexpr int BK = decltype(bk)::value;
    const auto kernel = K % BK ? mx_matmul_tile_kernel<decltype(afmt)::value, BM, BN, BK, decltype(ring)::value, false>
                               : mx_matmul_tile_kernel<decltype(afmt)::value, BM, BN, BK, decltype(ring)::value, true>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((long long)((M + BM - 1) / BM) * ((N + BN - 1) / BN))), dim3(kThreads), 0, s,
                       M, N, K, a_codes, a_scales, w_codes, w_scales, y, out_dtype);
  };
  auto sized = [&](auto afmt) {
    // Small batches are bound by W's bytes and go to the rows kernel, others to the largest tile of which there are
    // enough to give most compute units one. Where that is less than 64 x 64, tiles split among the waves are the
    // faster ones as long as every compute unit takes at most one. us at N = K = 4096, e2m1 rows / e4m3 rows, to bf16:
    //   M      rows          32 x 32, split  32 x 64, split  32 x 32       64 x 64       64 x 128      128 x 128     256 x 256
    //   16     4.4 / 5.5                                     5.8 / 9.7     7.8
    //   17     4.7 / 6.7     5.1 / 7.3       5.4 / 9.2
    //   32     5.6 / 7.9     5.3 / 7.1       5.7 / 9.0       5.6 / 9.6     7.5
    //   64     8.2 / 15.0    5.7 / 7.7       6.0 / 9.4       5.8 / 10.2    8.0 / 14.3    10.7
    //   128    14.0 / 32.7   7.7 / 13.3      6.5 / 10.1      7.4 / 13.0    8.6 / 14.6    11.9 / 19.6
    //   256                  13.4 / 24.5     11.6 / 18.2     11.9 / 21.7   9.1 / 15.2    12.2 / 19.7   15.4 / 33.5
    //   512                                                  20.4 / 36.4   13.3 / 27.2   12.7 / 20.7   16.1 / 34.6   32.8 / 81.3
    //   1024                                                               23.8 / 52.5   23.1 / 37.8   17.0 / 35.9   33.7 / 81.6
    //   2048                                                               44.1 / 103    43.7 / 73.5   30.4 / 66.6   35.3 / 83.5
    //   8192                                                               172 / 409     176 / 288     116 / 258     82 / 187
    // (An fp32 result of e4m3 rows takes up to 5% more.) Reductions below 256 go to the rows kernel: M = 8192, N =
    // 4096, e4m3 rows to bf16 442 us with K = 32, 457 with 224, where y's bytes alone would take 13.
    constexpr bool four = decltype(afmt)::value == kE2M1;
    typedef std::integral_constant<int, four ? 256 : 128> BK;
    typedef std::integral_constant<int, four ? 4 : 3> Ring;
    typedef std::integral_constant<int, 32> I32;
    typedef std::integral_constant<int, 64> I64;
    typedef std::integral_constant<int, 128> I128;
    typedef std::integral_constant<int, 256> I256;
    typedef std::integral_constant<int, 4> I4;
    auto enough = [&](int bm, int bn) { return (long long)((M + bm - 1) / bm) * ((N + bn - 1) / bn) >= 192; };
    auto few = [&](int bm, int bn) { return (long long)((M + bm - 1) / bm) * ((N + bn - 1) / bn) <= 256; };
    if (M > 32 && K >= 256) {
      if (enough(256, 256)) {
        const auto kernel = K % BK::value ? mx_matmul_wide_kernel<decltype(afmt)::value, false> : mx_matmul_wide_kernel<decltype(afmt)::value, true>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)((long long)((M + 255) / 256) * ((N + 255) / 256))), dim3(kWideThreads), 0, s, M, N, K,
                           a_codes, a_scales, w_codes, w_scales, y, out_dtype);
        return;
      }
      if (enough(128, 128)) return tiles(afmt, I128(), I128(), BK(), I4());
      if (enough(64, 128)) return tiles(afmt, I64(), I128(), I256(), Ring());
      if (enough(64, 64)) return tiles(afmt, I64(), I64(), I256(), I4());
    }
    if ((M > 32 || (M > 16 && !four)) && K >= 256) {
      if (few(32, 32)) return split(afmt, I32(), I32(), std::integral_constant<int, four ? 2 : 3>());
      if (few(32, 64)) return split(afmt, I32(), I64(), std::integral_constant<int, four ? 3 : 2>());
      if (M > 32) return tiles(afmt, I32(), I32(), I256(), I4());
    }
    if (M <= 16) go(afmt, std::integral_constant<int, 1>());
    else if (M <= 32) go(afmt, std::integral_constant<int, 2>());
    else go(afmt, std::integral_constant<int, 4>());
  };
  if (a_format == kE2M1) sized(std::integral_constant<int, kE2M1>());
  else sized(std::integral_constant<int, kE4M3>());
  return hipGetLastError();
}

}  // namespace moew2
