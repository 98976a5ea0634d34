// The weight gradient of an expert's product in 8-bit floating point:
// D[g] = sum over the tokens of expert g of a[m][t] b[n][t], both operands
// quantised along the tokens with one power-of-two scale for each row and
// 128 tokens. The scales go into CDNA4's scaled matrix instruction as
// exponent bytes, so its fp32 accumulator holds the true sum over all tokens
// and no vector instruction touches it before the final rounding to bf16.

#include <vector>

#include "elem.h"
#include "internal.h"

namespace fp8g {
namespace {

using namespace elem;

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// Quantisation along the tokens, written transposed.
//
// A workgroup takes 128 tokens x 128 columns: thread (cg, rg) holds CV = 16
// bytes of columns and the 64 / CV consecutive tokens from rg 64 / CV on, so that
// its codes of one column are consecutive bytes of the transposed row. The
// codes cross the workgroup through LDS and leave as whole 128-byte rows.
// HBM-bound: sizeof(T) bytes in and one out per element.

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

// Two codes from two values that are at most FP8max in magnitude, or NaN or
// infinite; see the header for what those become.
template <int FMT>
__device__ __forceinline__ uint32_t code_pair(float x, float y) {
  uint32_t w;
  if constexpr (FMT == FMT_E4M3)
    w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, y, 0, false) & 0xFFFFu;
  else
    w = (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(x, y, 0, false) & 0xFFFFu;
  const float lim = FMT == FMT_E4M3 ? 448.0f : 57344.0f;
  if (__builtin_expect(!(__builtin_fabsf(x) <= lim) || !(__builtin_fabsf(y) <= lim), 0)) {
    const uint32_t inf = FMT == FMT_E4M3 ? 0x7Fu : 0x7Cu;
    const uint32_t sx = (__float_as_uint(x) >> 24) & 0x80u, sy = (__float_as_uint(y) >> 24) & 0x80u;
    if (x != x) w = (w & 0xFF00u) | sx | 0x7Fu;
    else if (!(__builtin_fabsf(x) <= lim)) w = (w & 0xFF00u) | sx | inf;
    if (y != y) w = (w & 0xFFu) | (sy | 0x7Fu) << 8;
    else if (!(__builtin_fabsf(y) <= lim)) w = (w & 0xFFu) | (sy | inf) << 8;
  }
  return w;
}

template <typename T, int FMT>
__global__ void __launch_bounds__(QTHREADS)
quant_transpose_kernel(const T* __restrict__ x, int64_t rows, int64_t cols, int64_t ldx, int vec,
                       uint8_t* __restrict__ qt, int64_t ldq, uint8_t* __restrict__ st) {
  constexpr int CV = 16 / (int)sizeof(T);              // columns of a thread
  constexpr int CG = QCOLS / CV;                       // column groups
  constexpr int RT = 64 / CV;                          // tokens of a thread
  constexpr int RG = QTHREADS / CG;                    // token groups (RG * RT = 128)
  static_assert(RG * RT == 128, "128 tokens");
  __shared__ float part[QTHREADS / 64][QCOLS];
  __shared__ __attribute__((aligned(16))) uint8_t tile[QCOLS * 128];
  const int cg = threadIdx.x % CG, rg = threadIdx.x / CG;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c0 = (int64_t)blockIdx.x * QCOLS + cg * CV;
  const int64_t r0 = (int64_t)blockIdx.y * 128 + rg * RT;
  const bool has = c0 < cols;                          // (cols % 16 == 0: all CV or none)
  float v[RT][CV];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const bool in = has && r0 + i < rows;
    const T* p = x + (r0 + i) * ldx + c0;
    if (in && vec) {
      const Pack<T, CV> w = *reinterpret_cast<const Pack<T, CV>*>(p);
#pragma unroll
      for (int c = 0; c < CV; ++c) v[i][c] = to_f32(w.v[c]);
    } else {
#pragma unroll
      for (int c = 0; c < CV; ++c) v[i][c] = in ? to_f32(p[c]) : 0.0f;
    }
  }
  // amax over the finite elements of each column
  float m[CV];
#pragma unroll
  for (int c = 0; c < CV; ++c) {
    m[c] = 0.0f;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const float y = __builtin_fabsf(v[i][c]);
      m[c] = __builtin_fmaxf(m[c], y < __builtin_inff() ? y : 0.0f);
    }
#pragma unroll
    for (int o = CG; o < 64; o <<= 1) m[c] = __builtin_fmaxf(m[c], __shfl_xor(m[c], o));
    if (lane < CG) part[wave][cg * CV + c] = m[c];
  }
  __syncthreads();
  // one piece (RT codes of a column) per column; piece p of a row lies at
  // p ^ (its column group's low bits), which spreads the lanes' writes over
  // the banks
  constexpr int PIECES = 128 / RT;
#pragma unroll
  for (int c = 0; c < CV; ++c) {
    const int col = cg * CV + c;
    const float top = __builtin_fmaxf(__builtin_fmaxf(part[0][col], part[1][col]),
                                      __builtin_fmaxf(part[2][col], part[3][col]));
    const int e = block_exponent<FMT>(top);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    uint32_t w[RT / 4];
#pragma unroll
    for (int i = 0; i < RT / 4; ++i)
      w[i] = code_pair<FMT>(v[4 * i][c] * down, v[4 * i + 1][c] * down) |
             code_pair<FMT>(v[4 * i + 2][c] * down, v[4 * i + 3][c] * down) << 16;
    uint32_t* to = reinterpret_cast<uint32_t*>(tile + col * 128 + ((rg ^ cg) % PIECES) * RT);
#pragma unroll
    for (int i = 0; i < RT / 4; ++i) to[i] = w[i];
    if (rg == 0 && has) st[(int64_t)blockIdx.y * cols + c0 + c] = (uint8_t)(e + 127);
  }
  __syncthreads();
  // 16 bytes per thread and step: eight lanes to a row
#pragma unroll
  for (int q = 0; q < QCOLS * 128 / (16 * QTHREADS); ++q) {
    const int i = q * QTHREADS + threadIdx.x;
    const int col = i >> 3, b16 = i & 7;
    const int g = col / CV;
    if ((int64_t)blockIdx.x * QCOLS + col >= cols) continue;
    Pack<uint32_t, 4> o;
#pragma unroll
    for (int h = 0; h < 16 / RT; ++h) {
      const int piece = (b16 * (16 / RT) + h) ^ (g % PIECES);
      const uint32_t* from = reinterpret_cast<const uint32_t*>(tile + col * 128 + piece * RT);
#pragma unroll
      for (int d = 0; d < RT / 4; ++d) o.v[h * (RT / 4) + d] = from[d];
    }
    *reinterpret_cast<Pack<uint32_t, 4>*>(qt + ((int64_t)blockIdx.x * QCOLS + col) * ldq +
                                          (int64_t)blockIdx.y * 128 + b16 * 16) = o;
  }
}

// ---------------------------------------------------------------------------
// The product. 128x128 tiles, four waves of 64x64; each K step (128 tokens)
// goes through registers into LDS.

constexpr int BT = 128;
constexpr int ROWB = 128 + 16;                         // LDS row: 128 codes, padded

__device__ __forceinline__ v8i frag(const uint8_t* p) {
  const uint4 lo = *reinterpret_cast<const uint4*>(p);
  const uint4 hi = *reinterpret_cast<const uint4*>(p + 16);
  v8i f;
  f[0] = (int)lo.x; f[1] = (int)lo.y; f[2] = (int)lo.z; f[3] = (int)lo.w;
  f[4] = (int)hi.x; f[5] = (int)hi.y; f[6] = (int)hi.z; f[7] = (int)hi.w;
  return f;
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

template <int FA, int FB>
__global__ void __launch_bounds__(256)
wgrad_kernel(WgradArgs a, int mblocks, int nblocks) {
  __shared__ __attribute__((aligned(16))) uint8_t la[BT * ROWB], lb[BT * ROWB];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  const int64_t tile = blockIdx.x;
  const int g = (int)(tile / ((int64_t)mblocks * nblocks));
  const int in_g = (int)(tile - (int64_t)g * mblocks * nblocks);
  const int64_t m0 = (int64_t)(in_g % mblocks) * BT, n0 = (int64_t)(in_g / mblocks) * BT;
  int kb0, kb1;
  token_blocks(a, g, kb0, kb1);
  v4f acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int kb = kb0; kb < kb1; ++kb) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = q * 256 + (int)threadIdx.x, r = i >> 3, c = (i & 7) * 16;
      const int64_t ra = min(m0 + r, a.M - 1), rb = min(n0 + r, a.N - 1);
      *reinterpret_cast<uint4*>(la + r * ROWB + c) =
          *reinterpret_cast<const uint4*>(a.a + ra * a.lda + (int64_t)kb * 128 + c);
      *reinterpret_cast<uint4*>(lb + r * ROWB + c) =
          *reinterpret_cast<const uint4*>(a.b + rb * a.ldb + (int64_t)kb * 128 + c);
    }
    int sa[4], sb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sa[i] = a.sa[(int64_t)kb * a.M + min(m0 + wm + i * 16 + (lane & 15), a.M - 1)];
      sb[i] = a.sb[(int64_t)kb * a.N + min(n0 + wn + i * 16 + (lane & 15), a.N - 1)];
    }
    __syncthreads();
    v8i fa[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      fa[i] = frag(la + (wm + i * 16 + (lane & 15)) * ROWB + (lane >> 4) * 32);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const v8i fb = frag(lb + (wn + j * 16 + (lane & 15)) * ROWB + (lane >> 4) * 32);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa[i], acc[i][j], FB, FA, 0,
                                                                     sb[j], 0, sa[i]);
    }
  }
  // (b first: lane l holds row l & 15 of the tile, columns 4 (l >> 4) .. +3)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + wm + i * 16 + (lane & 15);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + wn + j * 16 + (lane >> 4) * 4;
      if (m < a.M && n < a.N) {
        Pack<bf16_t, 4> o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o.v[e] = from_f32<bf16_t>(acc[i][j][e]);
        *reinterpret_cast<Pack<bf16_t, 4>*>(a.d + ((int64_t)g * a.M + m) * a.N + n) = o;
      }
    }
  }
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

typedef void (*WgradFn)(WgradArgs, int, int);
WgradFn wgrad_pick(int fa, int fb) {
  if (fa == FMT_E4M3) return fb == FMT_E4M3 ? wgrad_kernel<0, 0> : wgrad_kernel<0, 1>;
  return fb == FMT_E4M3 ? wgrad_kernel<1, 0> : wgrad_kernel<1, 1>;
}

}  // namespace

hipError_t launch_quantize_transpose(const void* x, int type, int64_t rows, int64_t cols,
                                     int64_t ldx, int fmt, uint8_t* qt, int64_t ldq, uint8_t* st,
                                     hipStream_t stream) {
  if (type == TYPE_F32) return quant_launch<float>(x, rows, cols, ldx, fmt, qt, ldq, st, stream);
  if (type == TYPE_BF16) return quant_launch<bf16_t>(x, rows, cols, ldx, fmt, qt, ldq, st, stream);
  return quant_launch<f16_t>(x, rows, cols, ldx, fmt, qt, ldq, st, stream);
}

hipError_t launch_wgrad(const WgradArgs& args, int fmt_a, int fmt_b, const DeviceInfo&,
                        hipStream_t stream) {
  const int64_t mblocks = (args.M + BT - 1) / BT, nblocks = (args.N + BT - 1) / BT;
  wgrad_pick(fmt_a, fmt_b)<<<dim3((unsigned)(mblocks * nblocks * args.G)), dim3(256), 0, stream>>>(
      args, (int)mblocks, (int)nblocks);
  return hipGetLastError();
}

void wgrad_kernels(std::vector<const void*>& out) {
  for (int fmt : {FMT_E4M3, FMT_E5M2}) {
    out.push_back((const void*)quant_kernel<float>(fmt));
    out.push_back((const void*)quant_kernel<bf16_t>(fmt));
    out.push_back((const void*)quant_kernel<f16_t>(fmt));
    for (int fb : {FMT_E4M3, FMT_E5M2}) out.push_back((const void*)wgrad_pick(fmt, fb));
  }
}

}  // namespace fp8g
