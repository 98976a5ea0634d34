// The weight gradient of an expert's product in 8-bit floating point:
// D[g] = sum over the tokens of expert g of a[m][t] b[n][t], both operands
// quantised along the tokens with one power-of-two scale for each row and
// 128 tokens. The scales go into CDNA4's scaled matrix instruction as
// exponent bytes, so its fp32 accumulator holds the true sum over all tokens
// and no vector instruction touches it before the final rounding to bf16.

#include <type_traits>
#include <vector>

#include "elem.h"
#include "gemm_index.h"
#include "internal.h"

namespace fp8g {
namespace {

using namespace elem;

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// Quantisation along the tokens, written transposed.
//
// A workgroup takes 128 tokens x 128 columns: thread (cg, rg) holds CV = 16
// bytes of columns and the 64 / CV consecutive tokens from rg 64 / CV on, so that
// its codes of one column are consecutive bytes of the transposed row. The
// codes cross the workgroup through LDS and leave as whole 128-byte rows.
// HBM-bound: sizeof(T) bytes in and one out per element. 4096x8192 bf16 23.2 us
// (4.3 TB/s), 4864x4096 12.3 us (4.9), 4096x8192 fp32 35.8 us (4.7). With the values
// widened to fp32 in registers, and each code compared and packed on its own, 30.3
// us (bf16); 256 tokens x 64 columns per workgroup were slower than 128 x 128.

constexpr int QTHREADS = 256;
constexpr int QCOLS = 128;

// e = ceil(log2(amax / FP8max)) held to [-126, 126]; FP8max = 1.75 2^EMAX.
template <int FMT>
__device__ __forceinline__ int block_exponent(float amax) {
  constexpr int EMAX = FMT == FMT_E4M3 ? 8 : 15;
  const uint32_t u = __float_as_uint(amax);
  // (a subnormal amax has exponent field 0 and ends at the lower bound)
  int e = (int)(u >> 23) - 127 - EMAX + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -126 ? -126 : (e > 126 ? 126 : e);
  return amax > 0.0f ? e : 0;
}

// Code of x 2^-e for an x that may be NaN or infinite.
template <int FMT>
__device__ __forceinline__ uint32_t code_any(float x, float down) {
  const uint32_t sign = (__float_as_uint(x) >> 24) & 0x80u;
  if (x != x) return sign | 0x7Fu;
  if (__builtin_fabsf(x) == __builtin_inff()) return sign | (FMT == FMT_E4M3 ? 0x7Fu : 0x7Cu);
  const float y = x * down;
  if constexpr (FMT == FMT_E4M3)
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, y, 0, false) & 0xFFu;
  else
    return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(y, y, 0, false) & 0xFFu;
}

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef bf16_t bf16x2 __attribute__((ext_vector_type(2)));
typedef f16_t f16x2 __attribute__((ext_vector_type(2)));

// What the quantiser does with 16 bytes of a row (W words of 32 bits, each
// one fp32 or two 16-bit values). Magnitudes are compared as integers, two
// 16-bit ones at a time. Adding BUMP to a magnitude's bits takes NaN and
// infinity over the sign bit, below every finite value in a signed maximum.
// Codes: gfx950 converts two values, divided by a power of two, at once and
// rounds to nearest even; the values are finite there.
template <typename T>
struct Row16;
template <>
struct Row16<float> {
  static constexpr int PER = 1;                        // values in a word
  static constexpr uint32_t BUMP = 0x00800000u, TOP = 0x7F800000u;
  __device__ static __forceinline__ uint32_t mag(uint32_t w) { return w & 0x7FFFFFFFu; }
  __device__ static __forceinline__ uint32_t max_any(uint32_t a, uint32_t b) { return a > b ? a : b; }
  __device__ static __forceinline__ uint32_t max_finite(uint32_t a, uint32_t b) {
    return (int)a > (int)b ? a : b;
  }
  __device__ static __forceinline__ uint32_t bump(uint32_t m) { return m + BUMP; }
  __device__ static __forceinline__ uint32_t field(uint32_t w, int) { return w; }
  __device__ static __forceinline__ float value(uint32_t w, int) { return __uint_as_float(w); }
  // codes of a column's values in words a and b into one half of `old`
  template <int FMT, bool HI>
  __device__ static __forceinline__ uint32_t codes(uint32_t old, uint32_t a, uint32_t b, int,
                                                   float scale) {
    const s16x2 o = __builtin_bit_cast(s16x2, old);
    const float x = __uint_as_float(a), y = __uint_as_float(b);
    if constexpr (FMT == FMT_E4M3)
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, x, y, scale, HI));
    else
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(o, x, y, scale, HI));
  }
};
template <typename T>
struct Row16 {
  static constexpr int PER = 2;
  static constexpr uint32_t TOP = std::is_same<T, bf16_t>::value ? 0x7F80u : 0x7C00u;
  static constexpr uint32_t BUMP = (0x8000u - TOP) * 0x10001u;
  __device__ static __forceinline__ uint32_t mag(uint32_t w) { return w & 0x7FFF7FFFu; }
  __device__ static __forceinline__ uint32_t max_any(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
  }
  __device__ static __forceinline__ uint32_t max_finite(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(s16x2, a),
                                                                  __builtin_bit_cast(s16x2, b)));
  }
  __device__ static __forceinline__ uint32_t bump(uint32_t m) {
    return __builtin_bit_cast(uint32_t,
                              __builtin_bit_cast(u16x2, m) + __builtin_bit_cast(u16x2, BUMP));
  }
  __device__ static __forceinline__ uint32_t field(uint32_t w, int h) {
    return h ? w >> 16 : w & 0xFFFFu;
  }
  __device__ static __forceinline__ float value(uint32_t w, int h) {
    return to_f32(__builtin_bit_cast(T, (uint16_t)field(w, h)));
  }
  template <int FMT, bool HI>
  __device__ static __forceinline__ uint32_t codes(uint32_t old, uint32_t a, uint32_t b, int h,
                                                   float scale) {
    const s16x2 o = __builtin_bit_cast(s16x2, old);
    // (bytes 0, 1 or 2, 3 of a, then the same of b)
    const uint32_t w = __builtin_amdgcn_perm(b, a, h ? 0x07060302u : 0x05040100u);
    s16x2 r;
    if constexpr (std::is_same<T, bf16_t>::value) {
      const bf16x2 v = __builtin_bit_cast(bf16x2, w);
      if constexpr (FMT == FMT_E4M3) r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, v, scale, HI);
      else r = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(o, v, scale, HI);
    } else {
      const f16x2 v = __builtin_bit_cast(f16x2, w);
      if constexpr (FMT == FMT_E4M3) r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(o, v, scale, HI);
      else r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(o, v, scale, HI);
    }
    return __builtin_bit_cast(uint32_t, r);
  }
};

template <typename T, int FMT>
__global__ void __launch_bounds__(QTHREADS)
quant_transpose_kernel(const T* __restrict__ x, int64_t rows, int64_t cols, int64_t ldx, int vec,
                       uint8_t* __restrict__ qt, int64_t ldq, uint8_t* __restrict__ st) {
  using R = Row16<T>;
  constexpr int PER = R::PER;                          // values in a 32-bit word
  constexpr int CV = 4 * PER;                          // columns of a thread
  constexpr int CG = QCOLS / CV;                       // column groups
  constexpr int RT = 64 / CV;                          // tokens of a thread
  static_assert(QTHREADS / CG * RT == 128, "128 tokens");
  __shared__ uint32_t part[QTHREADS / 64][CG][4];
  __shared__ __attribute__((aligned(16))) uint8_t tile[QCOLS * 128];
  const int cg = threadIdx.x % CG, rg = threadIdx.x / CG;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * QCOLS + cg * CV;
  const int64_t r0 = (int64_t)blockIdx.y * 128 + rg * RT;
  const bool has = c0 < cols;                          // (cols % 16 == 0: all CV or none)
  uint4 v[RT];
  const T* p = x + r0 * ldx + c0;
  if (vec && has && r0 + RT <= rows) {
#pragma unroll
    for (int i = 0; i < RT; ++i) v[i] = *reinterpret_cast<const uint4*>(p + i * ldx);
  } else {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      Pack<T, CV> w;
#pragma unroll
      for (int c = 0; c < CV; ++c) w.v[c] = has && r0 + i < rows ? p[i * ldx + c] : (T)0.0f;
      v[i] = __builtin_bit_cast(uint4, w);
    }
  }
  const auto word = [](const uint4& u, int k) { return k == 0 ? u.x : k == 1 ? u.y : k == 2 ? u.z : u.w; };
  // amax of each column over the finite values of all tokens, and the largest magnitude
  // among this thread's own, NaN and infinity on top
  uint32_t any[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t m = R::BUMP;
    any[k] = 0u;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const uint32_t y = R::mag(word(v[i], k));
      any[k] = R::max_any(any[k], y);
      m = R::max_finite(m, R::bump(y));
    }
#pragma unroll
    for (int o = CG; o < 64; o <<= 1) m = R::max_finite(m, (uint32_t)__shfl_xor((int)m, o));
    if (lane < CG) part[wave][cg][k] = m;
  }
  __syncthreads();
  // a piece is RT codes of a column; piece q of a row lies at q ^ (its column
  // group), which spreads the lanes' writes over the banks
  constexpr int PIECES = 128 / RT;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t top = R::max_finite(R::max_finite(part[0][cg][k], part[1][cg][k]),
                                       R::max_finite(part[2][cg][k], part[3][cg][k]));
#pragma unroll
    for (int h = 0; h < PER; ++h) {
      const int col = cg * CV + k * PER + h;
      const uint32_t bits = R::field(top, h) - R::field(R::BUMP, h);
      const int e = block_exponent<FMT>(R::value(PER == 2 ? bits << (16 * h) : bits, h));
      const float scale = __uint_as_float((uint32_t)(127 + e) << 23);
      uint32_t w[RT / 4];
#pragma unroll
      for (int i = 0; i < RT / 4; ++i) {
        w[i] = R::template codes<FMT, false>(0u, word(v[4 * i], k), word(v[4 * i + 1], k), h, scale);
        w[i] = R::template codes<FMT, true>(w[i], word(v[4 * i + 2], k), word(v[4 * i + 3], k), h, scale);
      }
      if (__builtin_expect(R::field(any[k], h) >= R::TOP, 0)) {
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < RT / 4; ++i) {
          w[i] = 0u;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w[i] |= code_any<FMT>(R::value(word(v[4 * i + q], k), h), down) << (8 * q);
        }
      }
      uint32_t* to = reinterpret_cast<uint32_t*>(tile + col * 128 + ((rg ^ cg) % PIECES) * RT);
#pragma unroll
      for (int i = 0; i < RT / 4; ++i) to[i] = w[i];
      if (rg == 0 && has) st[(int64_t)blockIdx.y * cols + c0 + k * PER + h] = (uint8_t)(e + 127);
    }
  }
  __syncthreads();
  // 16 bytes per thread and step: eight lanes to a row
#pragma unroll
  for (int q = 0; q < QCOLS * 128 / (16 * QTHREADS); ++q) {
    const int i = q * QTHREADS + threadIdx.x;
    const int col = i >> 3, b16 = i & 7;
    if ((int64_t)blockIdx.x * QCOLS + col >= cols) continue;
    Pack<uint32_t, 4> o;
#pragma unroll
    for (int h = 0; h < 16 / RT; ++h) {
      const int piece = ((b16 * (16 / RT) + h) ^ (col / CV)) % PIECES;
      const uint32_t* from = reinterpret_cast<const uint32_t*>(tile + col * 128 + piece * RT);
#pragma unroll
      for (int d = 0; d < RT / 4; ++d) o.v[h * (RT / 4) + d] = from[d];
    }
    *reinterpret_cast<Pack<uint32_t, 4>*>(qt + ((int64_t)blockIdx.x * QCOLS + col) * ldq +
                                          (int64_t)blockIdx.y * 128 + b16 * 16) = o;
  }
}

// ---------------------------------------------------------------------------
// The product. Two kernels: 256x256 tiles where there are enough of them to fill the chip
// and they are full enough, 128x128 tiles otherwise. In both, codes go from global memory
// straight into LDS; each 128-byte LDS row holds one row's 128 tokens, its
// 16-byte chunks swizzled (swz).

typedef __attribute__((address_space(3))) void* lds_ptr_t;
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_ptr_t)p);
}
// Direct global -> LDS copies, through inline assembly so that the compiler
// does not wait for all of them before the next LDS read; the waits are
// explicit, before the barrier that publishes a stage.
__device__ __forceinline__ void copy16(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "{m0}"(lds)
               : "memory");
}
__device__ __forceinline__ void copy4(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "{m0}"(lds)
               : "memory");
}
constexpr int vmcnt_only(int n) { return (n & 0xF) | (0x7 << 4) | (0xF << 8) | (((n >> 4) & 3) << 14); }

// Chunk swizzle of an LDS row of 128 bytes (16-byte chunks): fragment reads
// of 8 or 16 consecutive rows meet every bank group equally.
__device__ __forceinline__ int swz(int row, int chunk) {
  return chunk ^ (row & 7) ^ ((row >> 3) & 1);
}

// Fragment f of a band of rows, tokens 64 kh .. +63: lane l holds position
// l % 32, tokens 32 (l / 32) .. +31 of those.
__device__ __forceinline__ v8i read_frag(const uint8_t* band, int f, int kh, int lane) {
  const int r = f * 32 + (lane & 31), c = kh * 4 + (lane >> 5) * 2;
  const uint4 lo = *reinterpret_cast<const uint4*>(band + r * 128 + swz(r, c) * 16);
  const uint4 hi = *reinterpret_cast<const uint4*>(band + r * 128 + swz(r, c + 1) * 16);
  v8i v;
  v[0] = (int)lo.x; v[1] = (int)lo.y; v[2] = (int)lo.z; v[3] = (int)lo.w;
  v[4] = (int)hi.x; v[5] = (int)hi.y; v[6] = (int)hi.z; v[7] = (int)hi.w;
  return v;
}

// Fragments j of b and i of a, whose exponents are bytes j and i of sb and
// sa. (i and j are constants where this is inlined.)
template <int FA, int FB>
__device__ __forceinline__ v16f mfma(const v8i& b, const v8i& a, const v16f& c, int j, uint32_t sb,
                                     int i, uint32_t sa) {
#define FP8G_M(J_, I_)                                                                          \
  case J_ * 4 + I_:                                                                             \
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, FB, FA, J_, (int)sb, I_,    \
                                                           (int)sa);
#define FP8G_M4(J_) FP8G_M(J_, 0) FP8G_M(J_, 1) FP8G_M(J_, 2) FP8G_M(J_, 3)
  switch (j * 4 + i) {
    FP8G_M4(0) FP8G_M4(1) FP8G_M4(2) FP8G_M4(3)
  }
#undef FP8G_M4
#undef FP8G_M
  return c;
}

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float x, float y) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
}

// The blocks of 128 tokens of expert g.
__device__ __forceinline__ void token_blocks(const WgradArgs& a, int g, int& kb0, int& kb1) {
  const int last = (int)(a.T / 128);
  if (!a.group) {
    kb0 = 0;
    kb1 = last;
    return;
  }
  const int lo = a.group[g], hi = a.group[g + 1];
  kb0 = lo < 0 ? 0 : min(lo / 128, last);
  kb1 = hi < 0 ? 0 : min(hi / 128, last);
}

// 128x128 tiles, four waves of 64x64, four LDS stages: a step's fragments are read
// during the one before, and its copies issued three and a half steps ahead, since
// with few workgroups a step's time is what its copies take to arrive. One barrier
// a step, half way: it publishes the stage that has landed and frees the one whose
// fragments are all in registers. One copy stands behind a matrix instruction, as in
// the large kernel. Position r of fragment i of a wave's 64 rows is row 2 r + i, so
// that a lane's exponents are two adjacent bytes and its results runs of 8 columns.
// Bound by latency: T 128 4.3 us, T 1024 7.6 to 8.5 us, T 4096 18 to 19 us (0.4 us a
// step, of which the copies' issue and the matrix instructions are 0.25 each) up to
// one workgroup per CU. With a step's copies, reads and products one after the other
// 4.3, 8.7 to 9.7 and 22 to 23 us; through registers and one LDS stage 13.4 us at T
// 1024. Runs of tiles per XCD are faster for some shapes and slower for others
// (T 4096, 1040x2064: 17.2 against 18.1 us, 2048x2048: 20.5 against 18.8).
constexpr int BT = 128;
constexpr int RING = 4;
constexpr int RSTAGE = 2 * BT * 128 + 2 * BT;
constexpr int RCOPIES = 9;                             // a wave's copies of a stage

template <int FA, int FB>
__global__ void __launch_bounds__(256, 1)
wgrad_ring_kernel(WgradArgs a, int mblocks, int nblocks) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[RING * RSTAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = mblocks * nblocks;
  const int g = (int)blockIdx.x / per, in_g = (int)blockIdx.x - g * per;
  const int64_t m0 = (int64_t)(in_g % mblocks) * BT, n0 = (int64_t)(in_g / mblocks) * BT;
  const int mv = (int)min((int64_t)BT, a.M - m0), nv = (int)min((int64_t)BT, a.N - n0);
  int kb0, kb1;
  token_blocks(a, g, kb0, kb1);
  const int steps = __builtin_amdgcn_readfirstlane(kb1 - kb0);
  // copies: waves 0 and 1 take a's two bands of 64 rows, 2 and 3 b's; copy c
  // is fragment c / 4, positions 8 (c % 4) .. +7; then 128 exponents (0 and 2 a's,
  // 1 and 3 b's)
  const uint8_t* const src = wave < 2 ? a.a + m0 * a.lda : a.b + n0 * a.ldb;
  const uint32_t ld = (uint32_t)(wave < 2 ? a.lda : a.ldb);
  const int last = (wave < 2 ? mv : nv) - 1, band = (wave & 1) * 64;
  const uint8_t* const esrc = (wave & 1) ? a.sb + n0 : a.sa + m0;
  const int64_t estep = (wave & 1) ? a.N : a.M;
  const uint32_t eoff = (uint32_t)min((lane & 31) * 4, ((wave & 1) ? nv : mv) - 4);
  uint32_t voff[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int row = band + ((c & 3) * 8 + (lane >> 3)) * 2 + (c >> 2);
    voff[c] = (uint32_t)min(row, last) * ld + (uint32_t)((lane & 7) ^ (lane >> 3) ^ (c & 1)) * 16u;
  }
  const uint32_t base = lds_addr(lds);
  // copy c of a step (past the end the last step's again, for nothing: every wait
  // counts alike)
  auto copy = [&](int s, int c) __attribute__((always_inline)) {
    const int64_t kb = kb0 + min(s, steps - 1);
    const uint32_t st = base + (uint32_t)(s % RING) * RSTAGE;
    if (c < 8) copy16(src + kb * 128, voff[c], st + (uint32_t)((wave >> 1) * BT + band + c * 8) * 128u);
    else if (lane < 32) copy4(esrc + kb * estep, eoff, st + 2 * BT * 128 + (wave & 1) * BT);
  };
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  const int ea = 2 * BT * 128 + wm + (lane & 31) * 2, eb = 2 * BT * 128 + BT + wn + (lane & 31) * 2;
  // own reads and copies of long enough ago have arrived; then everyone's have
  auto meet = [&](auto n) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_waitcnt(vmcnt_only(decltype(n)::value));
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  v16f acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = v16f{};
  if (steps > 0) {
#pragma unroll
    for (int c = 0; c < 3 * RCOPIES + 5; ++c) copy(c / RCOPIES, c % RCOPIES);
    meet(std::integral_constant<int, 2 * RCOPIES + 5>{});
    v8i fa[2][2], fb[2][2];                            // [fragment][half of the 128 tokens]
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i][h] = read_frag(lds + wm * 128, i, h, lane);
        fb[i][h] = read_frag(lds + BT * 128 + wn * 128, i, h, lane);
      }
    uint32_t sa = *reinterpret_cast<const uint16_t*>(lds + ea);
    uint32_t sb = *reinterpret_cast<const uint16_t*>(lds + eb);
    for (int s = 0; s < steps; ++s) {
      // (the empty asm keeps a pure instruction from moving to where it is used)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int i = m >> 1, j = m & 1;
        acc[i][j] = mfma<FA, FB>(fb[j][0], fa[i][0], acc[i][j], j, sb, i, sa);
        asm volatile("" : "+a"(acc[i][j]));
        copy(s + 3, 5 + m);
      }
      // this stage has been read by all, and the next one's copies have landed: those
      // of two steps may be on their way
      meet(std::integral_constant<int, 2 * RCOPIES>{});
      const uint8_t* const st = lds + ((s + 1) % RING) * RSTAGE;
      const uint32_t sa_n = *reinterpret_cast<const uint16_t*>(st + ea);
      const uint32_t sb_n = *reinterpret_cast<const uint16_t*>(st + eb);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int i = m >> 1, j = m & 1;
        if (i == 0) fa[j][0] = read_frag(st + wm * 128, j, 0, lane);
        else fb[j][0] = read_frag(st + BT * 128 + wn * 128, j, 0, lane);
        acc[i][j] = mfma<FA, FB>(fb[j][1], fa[i][1], acc[i][j], j, sb, i, sa);
        asm volatile("" : "+a"(acc[i][j]));
        copy(s + 4, m);
        if (m == 3) copy(s + 4, 4);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i][1] = read_frag(st + wm * 128, i, 1, lane);
        fb[i][1] = read_frag(st + BT * 128 + wn * 128, i, 1, lane);
      }
      sa = sa_n;
      sb = sb_n;
    }
    // (no copy may arrive after the workgroup's LDS is someone else's)
    __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
  }
  // b is the first operand: lane l holds position l % 32 of fragment i of a,
  // and of fragment j of b positions 8 t + 4 (l / 32) + e; column 2 position + j
  uint16_t* const d = a.d + ((int64_t)g * a.M + m0) * a.N + n0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = wm + (lane & 31) * 2 + i;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int col = wn + t * 16 + (lane >> 5) * 8;
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = bf16_pair(acc[i][0][4 * t + e], acc[i][1][4 * t + e]);
      if (row < mv && col < nv) *reinterpret_cast<u32x4*>(d + (int64_t)row * a.N + col) = v;
    }
  }
}

// ---------------------------------------------------------------------------
// 256x256 tiles: four waves of 128x128, one per SIMD, the 256 accumulators
// of a lane in the accumulation registers (nothing but the matrix unit
// touches them until the end, since the scales go into the instruction). Per
// 128 tokens a wave reads (128 + 128) x 128 bytes of LDS for 32 matrix
// instructions of 64 cycles: 64 bytes a cycle and CU, with the 32 of the
// copies into LDS three quarters of what the LDS moves; eight waves of
// 64x128 would need all of it.
//
// A workgroup walks tiles (expert, row block, column block); the 128-token
// steps of all its tiles form one sequence with two LDS stages. A step's 32
// matrix instructions:
//   0-15   fragments 0 and 1 of b against all of a. After the first four
//          everyone meets: a's part of this stage and b's first half have been read
//          by all (a step ahead), so that the copies of the step after next may
//          go there, and b's second half has landed and is read.
//   16-31  everyone meets again: this stage is read altogether, and the next
//          one's a and b first half have landed. Each fragment of a against 2
//          and 3 of b, after which the next step's fragment takes its place.
// At most one copy and two LDS reads stand between two matrix instructions: a
// copy holds its wave for about 58 cycles (the four waves of a CU share the
// path), which the 64 of a 32x32x64 instruction cover and the 32 of a
// 16x16x128 do not; copies in bursts leave the matrix unit waiting.
//
// Measured (T 4096, 8192x8192: 550 GFLOP; T 4096, 8 experts, 4096x7168: 470 MB of
// results), the kernel alone, repeated, random codes under one scale: first version,
// one barrier and three bursts of copies a step 215 and 209
// us; two meets, spread copies 205 and 205; 32x32x64, whole-line stores 197 and 166;
// a tile's first step from a zero operand 192 (2.9 PFLOP/s; the library's 8-bit
// product of 8192^3 reaches 3.06 here) and 158. On quantised normal data 206
// (2.67 PFLOP/s) and 164, since the clock that the chip holds goes by the data (beside the
// first 1.6 to 1.7 GHz, 1.8 on random codes; beside the second 1.8 to 1.9 and 2.0). Under the
// kernel trace 236 and 185.
// Before the last step, without copies 168 and 149, without stores 175 and 97,
// with neither 147 and 85: the large layer is bound by the copies' issue, the
// experts by writing 128 KB per tile after 2 to 15 steps, during which the matrix
// unit is idle and the next copies queue behind the stores. Prefetching into L2, operands laid out in tiles,
// fewer or more rows per XCD group and shifting the experts' order per XCD or
// CU changed nothing.
//
// Which global row lies in which LDS row is free, as each lane of a copy has
// its own address. The rows of a 128-row band are dealt so that
//   a: position r of fragment i is row 4 r + i: one 4-byte LDS read gives a
//      lane the exponent bytes of its four fragments;
//   b: position x of fragment j is row 4 col_of(x) + j: likewise, and a lane
//      ends up with runs of 8 adjacent columns of a row (see the store).

constexpr int TS = 256;                                // tile side
constexpr int STAGE = 2 * TS * 128 + 2 * TS;           // codes of a and b, then their exponent bytes
constexpr int COPIES = 17;                             // a wave's copies of a stage: 8 + 8, and one of exponents
constexpr int EARLY = 13;                              // those that are read a step ahead,
constexpr int EARLY_FIRST = 8;                         // of these, issued in a step's first half
constexpr int STORES = 32;                             // a wave's stores of a full tile
constexpr int MAX_G = 1024;

// The experts that have tokens, in order, and those that have none.
struct Experts {
  int full[MAX_G], kb0[MAX_G], steps[MAX_G];
  int empty[MAX_G];
  int nfull, nempty;
};

struct Tile {
  const uint8_t *a, *b, *sa, *sb;                      // first row, first token block
  uint16_t* d;
  int mv, nv, steps;                                   // rows and columns that exist
};

__device__ __forceinline__ void tile_of(const WgradArgs& a, const Experts& ex, int slot, int mblocks,
                                        int nblocks, Tile& t) {
  const int per = mblocks * nblocks;
  const int at = __builtin_amdgcn_readfirstlane(slot / per);
  int mb, nb;
  gidx::swizzle_tile(slot - at * per, mblocks, nblocks, 4, mb, nb);
  const int g = __builtin_amdgcn_readfirstlane(ex.full[at]);
  const int64_t kb0 = __builtin_amdgcn_readfirstlane(ex.kb0[at]);
  const int64_t m0 = (int64_t)mb * TS, n0 = (int64_t)nb * TS;
  t.steps = __builtin_amdgcn_readfirstlane(ex.steps[at]);
  t.mv = (int)min((int64_t)TS, a.M - m0);
  t.nv = (int)min((int64_t)TS, a.N - n0);
  t.a = a.a + m0 * a.lda + kb0 * 128;
  t.b = a.b + n0 * a.ldb + kb0 * 128;
  t.sa = a.sa + kb0 * a.M + m0;
  t.sb = a.sb + kb0 * a.N + n0;
  t.d = a.d + ((int64_t)g * a.M + m0) * a.N + n0;
}

// This lane's copy offsets for a tile. Wave w copies the LDS rows of band
// w / 2 whose bit 3 is w % 2: copy c of an operand is fragment c % 4, positions 16 (c / 4)
// + 8 (w % 2) .. +7. Rows past the tile's last are copies of it (read in
// bounds, never stored).
struct Plan {
  uint32_t va, ma, vb, mb;                             // copy 0's offset, the last row's
  uint32_t vs;
};
__device__ __forceinline__ int col_of(int x) {         // position of b -> column / 4
  return (x & 1) | ((x >> 2) & 1) << 1 | ((x >> 1) & 1) << 2 | (x >> 3) << 3;
}
__device__ __forceinline__ void make_plan(Plan& p, const WgradArgs& a, const Tile& t, int wave,
                                          int lane) {
  const int band = wave >> 1, h = wave & 1, r = h * 8 + (lane >> 3);
  const uint32_t ch = (uint32_t)((lane & 7) ^ (lane >> 3) ^ h) * 16u;
  p.va = (uint32_t)(band * 128 + r * 4) * (uint32_t)a.lda + ch;
  p.vb = (uint32_t)(band * 128 + col_of(r) * 4) * (uint32_t)a.ldb + ch;
  p.ma = (uint32_t)(t.mv - 1) * (uint32_t)a.lda + ch;
  p.mb = (uint32_t)(t.nv - 1) * (uint32_t)a.ldb + ch;
  p.vs = (uint32_t)min(lane * 4, (h ? t.nv : t.mv) - 4);
}

// Copy c of a wave's share of a stage: a's eight, b's fragments 0 and 1, the
// exponents (waves 0 and 2 a's, 1 and 3 b's, twice the same bytes), b's 2 and 3.
__device__ __forceinline__ void issue(const Plan& p, const WgradArgs& a, const Tile& t, int kb,
                                      uint32_t stage, int wave, int c) {
  const uint32_t dst = stage + (uint32_t)((wave >> 1) * 16 + (wave & 1)) * 1024u;
  // (opaque: formed at each copy, the 16 offsets would otherwise be kept in
  // registers that the fragments need)
  uint32_t lda = (uint32_t)a.lda, ldb = (uint32_t)a.ldb;
  asm volatile("" : "+s"(lda), "+s"(ldb));
  if (c < 8) {
    const int f = c & 3, half = c >> 2;
    copy16(t.a + (int64_t)kb * 128, min(p.va + (uint32_t)(f + 64 * half) * lda, p.ma),
           dst + (uint32_t)(f * 4096 + half * 2048));
  } else if (c == 12) {
    copy4((wave & 1) ? t.sb + (int64_t)kb * a.N : t.sa + (int64_t)kb * a.M, p.vs,
          stage + 2 * TS * 128 + (wave & 1) * TS);
  } else {
    const int q = c < 12 ? c - 8 : c - 9, f = q >> 1, half = q & 1;
    copy16(t.b + (int64_t)kb * 128, min(p.vb + (uint32_t)(f + 64 * half) * ldb, p.mb),
           dst + TS * 128 + (uint32_t)(f * 4096 + half * 2048));
  }
}

template <int FA, int FB>
__global__ void __launch_bounds__(256, 1)
wgrad_tile_kernel(WgradArgs a, int mblocks, int nblocks, int xcd_remap) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STAGE];
  __shared__ Experts ex;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grid = gridDim.x, w = blockIdx.x;
  if (wave == 0) {
    int nf = 0, ne = 0;
    for (int g0 = 0; g0 < a.G; g0 += 64) {
      const int g = g0 + lane;
      int kb0 = 0, kb1 = 0;
      if (g < a.G) token_blocks(a, g, kb0, kb1);
      const bool has = kb1 > kb0, none = g < a.G && !has;
      const uint64_t mf = __ballot(has), me = __ballot(none);
      const uint64_t below = (1ull << lane) - 1;
      if (has) {
        const int i = nf + __popcll(mf & below);
        ex.full[i] = g;
        ex.kb0[i] = kb0;
        ex.steps[i] = kb1 - kb0;
      }
      if (none) ex.empty[ne + __popcll(me & below)] = g;
      nf += __popcll(mf);
      ne += __popcll(me);
    }
    if (lane == 0) {
      ex.nfull = nf;
      ex.nempty = ne;
    }
  }
  __syncthreads();
  const int per = mblocks * nblocks;
  const int nfull = __builtin_amdgcn_readfirstlane(ex.nfull);
  const int nempty = __builtin_amdgcn_readfirstlane(ex.nempty);
  // experts without tokens: zeros, row by row
  for (int64_t r = w; r < (int64_t)nempty * a.M; r += grid) {
    const int g = ex.empty[r / a.M];
    uint16_t* row = a.d + ((int64_t)g * a.M + r % a.M) * a.N;
    for (int64_t n = threadIdx.x * 8; n < a.N; n += 256 * 8)
      __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, reinterpret_cast<u32x4*>(row + n));
  }
  const int tiles = nfull * per;
  const int first = xcd_remap ? (w & 7) * (grid >> 3) + (w >> 3) : w;
  if (first >= tiles) return;
  const int wm = wave >> 1, wn = wave & 1;
  const uint32_t base = lds_addr(lds);
  // copy cursor
  int p_slot = first, p_kb = 0;
  Tile tp;
  tile_of(a, ex, p_slot, mblocks, nblocks, tp);
  Plan pl;
  make_plan(pl, a, tp, wave, lane);
  auto advance = [&]() __attribute__((always_inline)) {
    // (past the last step it stays there: two stages are copied once more at
    // the end, for nothing, and every wait may count on the same copies)
    if (++p_kb == tp.steps) {
      if (p_slot + grid < tiles) {
        p_kb = 0;
        p_slot += grid;
        tile_of(a, ex, p_slot, mblocks, nblocks, tp);
        make_plan(pl, a, tp, wave, lane);
      } else {
        --p_kb;
      }
    }
  };
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int c = 0; c < COPIES; ++c) issue(pl, a, tp, p_kb, base + s * STAGE, wave, c);
    advance();
  }
  v16f acc[4][4];
  v8i af[4][2], bf[4][2];        // fragments of a and b, by halves of the 128 tokens
  uint32_t sa, sb, sa_n, sb_n;   // their exponent bytes
  const int pos = lane & 31;
  const int ea = 2 * TS * 128 + wm * 128 + pos * 4;
  const int eb = 2 * TS * 128 + TS + wn * 128 + col_of(pos) * 4;
  const int oa = wm * 128 * 128, ob = TS * 128 + wn * 128 * 128;
  __builtin_amdgcn_s_waitcnt(vmcnt_only(2 * COPIES - EARLY));
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      af[i][h] = read_frag(lds + oa, i, h, lane);
      if (i < 2) bf[i][h] = read_frag(lds + ob, i, h, lane);
    }
  sa = *reinterpret_cast<const uint32_t*>(lds + ea);
  sb = *reinterpret_cast<const uint32_t*>(lds + eb);

  // Two points of a step where everyone waits for copies and meets: for b's
  // late fragments of this step, and half way for the early part of the next.
  // N copies have been issued since those; for three points after a full tile
  // its stores are newer too. (Waits may be longer than needed, never shorter:
  // where a ragged tile stores less, its stores are waited for.)
  int fresh = 0;
  auto meet = [&](auto n) __attribute__((always_inline)) {
    constexpr int N = decltype(n)::value;
    __builtin_amdgcn_s_waitcnt(0xC07F);                // lgkmcnt(0): own reads have arrived
    if (fresh > 0) __builtin_amdgcn_s_waitcnt(vmcnt_only(N + STORES));
    else __builtin_amdgcn_s_waitcnt(vmcnt_only(N));
    --fresh;
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  int s = 0;            // step, over all tiles
  for (int slot = first; slot < tiles; slot += grid) {
    Tile tc;
    tile_of(a, ex, slot, mblocks, nblocks, tc);
    // A tile's first step starts its sums from a zero operand: as one loop, the 256
    // registers are cleared by as many writes before it (dense 196 against 192 us,
    // experts 166 against 158).
    auto step = [&](auto first_step) __attribute__((always_inline)) {
      constexpr bool FIRST = decltype(first_step)::value;
      const uint8_t* __restrict__ cur = lds + (s & 1) * STAGE;
      const uint8_t* __restrict__ nxt = lds + ((s & 1) ^ 1) * STAGE;
      const uint32_t stage = base + (s & 1) * STAGE;
      // (between two matrix instructions at most two reads and a copy, which
      // fit their 64 cycles: a run of them would leave the matrix unit waiting)
#define FP8G_MFMA(I_, J_, H_)                                                          \
  do {                                                                                 \
    const v16f c_ = FIRST && H_ == 0 ? v16f{} : acc[I_][J_];                           \
    acc[I_][J_] = mfma<FA, FB>(bf[J_][H_], af[I_][H_], c_, J_, sb, I_, sa);            \
    /* (a pure instruction: without this it is moved to where it is used) */           \
    asm volatile("" : "+a"(acc[I_][J_]));                                              \
  } while (0)
      // first half: fragments 0 and 1 of b, each against all of a
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        const int j = m >> 3, h = (m >> 2) & 1, i = m & 3;
        if (m == 4) meet(std::integral_constant<int, COPIES>{});
        if (m >= 4 && m < 8) bf[2 + ((m - 4) >> 1)][m & 1] = read_frag(cur + ob, 2 + ((m - 4) >> 1), m & 1, lane);
        FP8G_MFMA(i, j, h);
        if (m >= 4 && (m - 4) % 3 != 2) issue(pl, a, tp, p_kb, stage, wave, (m - 4) - (m - 4) / 3);
      }
      meet(std::integral_constant<int, COPIES - EARLY + EARLY_FIRST>{});
      // second half: each fragment of a against 2 and 3 of b, after which the
      // next step's takes its place
      sa_n = *reinterpret_cast<const uint32_t*>(nxt + ea);
      sb_n = *reinterpret_cast<const uint32_t*>(nxt + eb);
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        const int i = m >> 2, h = (m >> 1) & 1, j = 2 + (m & 1);
        if (m < 4) bf[m >> 1][m & 1] = read_frag(nxt + ob, m >> 1, m & 1, lane);
        FP8G_MFMA(i, j, h);
        if (m % 2 == 1) issue(pl, a, tp, p_kb, stage, wave, EARLY_FIRST + m / 2);
        if (m == 15) issue(pl, a, tp, p_kb, stage, wave, EARLY_FIRST + 8);
        // (the half of this fragment that is done with)
        if (m % 2 == 1) af[i][h] = read_frag(nxt + oa, i, h, lane);
      }
#undef FP8G_MFMA
      advance();
      sa = sa_n;
      sb = sb_n;
      ++s;
    };
    // (the sums stay where the matrix unit keeps them from here to the stores)
    auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[i][j]));
    };
    step(std::true_type{});
    pin();
#pragma nounroll
    for (int k = 1; k < tc.steps; ++k) step(std::false_type{});
    pin();
    const bool full = tc.mv == TS && tc.nv == TS;
    fresh = full ? 3 : 0;
    // A lane holds, of a's position pos, 16 positions of each fragment j of b:
    // for every t 8 adjacent columns (u = 0) and, 16 further, 8 more (u = 1);
    // the other half of the wave holds the 8 after each. Exchanging u = 1 of
    // lanes 0-15 (32-47) with u = 0 of lanes 16-31 (48-63) gives four lanes 64
    // bytes of a row, and exchanging t + 1 of lanes 0-7 of each 16 with t of
    // lanes 8-15 gives eight lanes its 128. Whole lines, non-temporal, eight
    // rows a store, measured fastest (16 rows x 64 bytes and 4 x 256 slower).
    const int l16 = lane & 15, q16 = lane >> 4;
    const int cl = wn * 128 + (l16 >> 3) * 32 + (q16 & 1) * 16 + (q16 >> 1) * 8;
    const int rl = wm * 128 + (l16 & 7) * 4;
    uint16_t* const d0 = tc.d + (int64_t)rl * a.N + cl;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int t2 = 0; t2 < 2; ++t2) {
        uint32_t v[2][2][4];                           // [t - 2 t2][u]
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int q = 4 * (2 * t2 + tt) + 2 * u + (w >> 1), j = (w & 1) * 2;
              v[tt][u][w] = bf16_pair(acc[i][j][q], acc[i][j + 1][q]);
            }
            const auto r = __builtin_amdgcn_permlane16_swap(v[tt][0][w], v[tt][1][w], false, false);
            v[tt][0][w] = r[0];
            v[tt][1][w] = r[1];
          }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          u32x4 lo, hi;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int x = (int)v[0][u][w], y = (int)v[1][u][w];
            lo[w] = (uint32_t)__builtin_amdgcn_update_dpp(x, y, 0x128, 0xF, 0xC, false);
            hi[w] = (uint32_t)__builtin_amdgcn_update_dpp(y, x, 0x128, 0xF, 0x3, false);
          }
          // positions (l16 & 7) + 16 u and 8 more of fragment i
          const int r0 = 64 * u + i, c = t2 * 64;
          const bool col = c + cl < tc.nv;
          if (full || (col && rl + r0 < tc.mv))
            __builtin_nontemporal_store(lo, reinterpret_cast<u32x4*>(d0 + (int64_t)r0 * a.N + c));
          if (full || (col && rl + r0 + 32 < tc.mv))
            __builtin_nontemporal_store(hi, reinterpret_cast<u32x4*>(d0 + (int64_t)(r0 + 32) * a.N + c));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // (no copy may arrive after the workgroup's LDS is someone else's)
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
}

template <typename T>
void (*quant_kernel(int fmt))(const T*, int64_t, int64_t, int64_t, int, uint8_t*, int64_t,
                              uint8_t*) {
  return fmt == FMT_E4M3 ? quant_transpose_kernel<T, FMT_E4M3>
                         : quant_transpose_kernel<T, FMT_E5M2>;
}

template <typename T>
hipError_t quant_launch(const void* x, int64_t rows, int64_t cols, int64_t ldx, int fmt,
                        uint8_t* qt, int64_t ldq, uint8_t* st, hipStream_t stream) {
  const int vec = (uintptr_t)x % 16 == 0 && ldx * (int64_t)sizeof(T) % 16 == 0;
  const dim3 grid((unsigned)((cols + QCOLS - 1) / QCOLS), (unsigned)((rows + 127) / 128));
  quant_kernel<T>(fmt)<<<grid, dim3(QTHREADS), 0, stream>>>((const T*)x, rows, cols, ldx, vec, qt,
                                                            ldq, st);
  return hipGetLastError();
}

typedef void (*TileFn)(WgradArgs, int, int, int);
TileFn tile_pick(int fa, int fb) {
  if (fa == FMT_E4M3) return fb == FMT_E4M3 ? wgrad_tile_kernel<0, 0> : wgrad_tile_kernel<0, 1>;
  return fb == FMT_E4M3 ? wgrad_tile_kernel<1, 0> : wgrad_tile_kernel<1, 1>;
}
typedef void (*RingFn)(WgradArgs, int, int);
RingFn ring_pick(int fa, int fb) {
  if (fa == FMT_E4M3) return fb == FMT_E4M3 ? wgrad_ring_kernel<0, 0> : wgrad_ring_kernel<0, 1>;
  return fb == FMT_E4M3 ? wgrad_ring_kernel<1, 0> : wgrad_ring_kernel<1, 1>;
}

}  // namespace

hipError_t launch_quantize_transpose(const void* x, int type, int64_t rows, int64_t cols,
                                     int64_t ldx, int fmt, uint8_t* qt, int64_t ldq, uint8_t* st,
                                     hipStream_t stream) {
  if (type == TYPE_F32) return quant_launch<float>(x, rows, cols, ldx, fmt, qt, ldq, st, stream);
  if (type == TYPE_BF16) return quant_launch<bf16_t>(x, rows, cols, ldx, fmt, qt, ldq, st, stream);
  return quant_launch<f16_t>(x, rows, cols, ldx, fmt, qt, ldq, st, stream);
}

hipError_t launch_wgrad(const WgradArgs& args, int fmt_a, int fmt_b, const DeviceInfo& dev,
                        hipStream_t stream) {
  const int64_t cus = dev.cu_count;
  const int64_t mb = (args.M + TS - 1) / TS, nb = (args.N + TS - 1) / TS, all = mb * nb * args.G;
  const int64_t mblocks = (args.M + BT - 1) / BT, nblocks = (args.N + BT - 1) / BT;
  const int64_t small = mblocks * nblocks * args.G;
  // 256x256 tiles when they are more than half the CUs; up to there, at most two
  // rounds of 128x128 tiles, whose copies are further ahead (dense, 128 against 256,
  // T 4096: 64 tiles of 256x256 18.8 / 38.7 us, 128 tiles 36.0 / 40.5, 140 tiles
  // 49.3 / 41.6, 256 tiles 67.2 / 48.7; T 1024: 64 tiles 8.8 / 16.2, 128 tiles 15.0 /
  // 16.3, 140 tiles 20.5 / 16.4). And only where 128x128 tiles need more rounds of
  // the CUs: many narrow experts leave most of a large tile empty (experts of T tokens,
  // rounds of 128 / of 256: 160 of T 128 64x64, 1 / 1, 4.2 / 8.1 us; 512 of T 128 128x128,
  // 2 / 2, 9.7 / 13.0; 160 of T 512 128x128, 1 / 1, 6.2 / 11.3; 160 of T 2048 384x128, 2 / 2, 44 / 48;
  // 160 of T 512 128x640, 4 / 2, 30.5 / 21.3; 400 of T 512 384x128, 5 / 4, 40.2 / 37.2; 64 of
  // T 512 528x528, 7 / 3, 36.3 / 31.7; but 33 of T 384 512x784, 4 / 2, 21.9 / 24.3).
  // (Also without tokens, where both only write zeros: the large kernel's grid has a
  // bound, and as many rounds are at most some hundred tiles more.)
  if (all > cus / 2 && (small + cus - 1) / cus > (all + cus - 1) / cus) {
    const int64_t grid = all < cus ? all : cus;
    tile_pick(fmt_a, fmt_b)<<<dim3((unsigned)grid), dim3(256), 0, stream>>>(
        args, (int)mb, (int)nb, grid % 8 == 0 ? 1 : 0);
    return hipGetLastError();
  }
  ring_pick(fmt_a, fmt_b)<<<dim3((unsigned)small), dim3(256), 0, stream>>>(args, (int)mblocks,
                                                                            (int)nblocks);
  return hipGetLastError();
}

void wgrad_kernels(std::vector<const void*>& out) {
  for (int fmt : {FMT_E4M3, FMT_E5M2}) {
    out.push_back((const void*)quant_kernel<float>(fmt));
    out.push_back((const void*)quant_kernel<bf16_t>(fmt));
    out.push_back((const void*)quant_kernel<f16_t>(fmt));
    for (int fb : {FMT_E4M3, FMT_E5M2}) {
      out.push_back((const void*)ring_pick(fmt, fb));
      out.push_back((const void*)tile_pick(fmt, fb));
    }
  }
}

}  // namespace fp8g
