// Products in 8-bit integers: the quantiser (one scale a row) and the product with a
// scale for each token and each output channel, dense and for every expert of a layer.
//
// d[m][n] = bf16( (fl32(sum_k a[m][k] b[n][k]) sa[m]) sb[n] ). The sum is a whole number,
// exact in 32 bits up to K = 131071 (codes -128 .. 127: K 2^14 < 2^31), so its order does
// not matter and every way of cutting the work gives the same bits.

#include <type_traits>
#include <vector>

#include "elem.h"
#include "internal.h"

namespace fp8g {
namespace {

using namespace elem;

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// Quantiser: scale = amax / 127, code = rne(fl32(x fl32(127 / amax))), both divisions
// correctly rounded and once a row. |x inv| <= 127 (1 + 2^-23), which rounds to 127. Below
// 2^-120 127 / amax would leave fp32's range: such a row counts as zero (scale and codes
// 0). A row with an infinity or NaN has the scale NaN and codes 0, so that every result of
// it is NaN.
constexpr int QTHREADS = 256;
constexpr float TINY_ROW = 0x1p-120f;

struct RowScale {
  float inv, scale;
  uint32_t keep;                                       // 0: the codes are zeros
};
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  const float amax = __uint_as_float(amax_bits);
  RowScale r;
  const bool bad = amax_bits >= 0x7F800000u, zero = amax < TINY_ROW;
  r.keep = bad || zero ? 0u : 0xFFFFFFFFu;
  r.inv = r.keep ? 127.0f / amax : 0.0f;
  r.scale = bad ? __builtin_nanf("") : (zero ? 0.0f : amax / 127.0f);
  return r;
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The code in the low byte: adding 1.5 2^23 rounds to a whole number, whose two's
// complement the low bits then hold.
__device__ __forceinline__ uint32_t code_bits(float x, float inv) {
#pragma clang fp contract(off)
  const float y = x * inv;
  return __float_as_uint(y + 12582912.0f);
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, const RowScale& r) {
  const uint32_t lo = __builtin_amdgcn_perm(code_bits(b, r.inv), code_bits(a, r.inv), 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm(code_bits(d, r.inv), code_bits(c, r.inv), 0x04000C0Cu);
  return (lo | hi) & r.keep;
}

template <typename T, int W>
__device__ __forceinline__ Pack<T, W> load_pack(const T* __restrict__ row, int64_t at, bool vec) {
  if (vec) return *reinterpret_cast<const Pack<T, W>*>(row + at);
  Pack<T, W> p;
#pragma unroll
  for (int w = 0; w < W; ++w) p.v[w] = row[at + w];
  return p;
}
template <typename T, int W>
__device__ __forceinline__ uint32_t pack_amax(const Pack<T, W>& p, uint32_t m) {
#pragma unroll
  for (int w = 0; w < W; ++w) m = max(m, abs_bits(to_f32(p.v[w])));
  return m;
}
template <typename T, int W>
__device__ __forceinline__ void store_codes(const Pack<T, W>& p, const RowScale& r, int8_t* q) {
  Pack<uint32_t, W / 4> o;
#pragma unroll
  for (int w = 0; w < W; w += 4)
    o.v[w / 4] = codes4(to_f32(p.v[w]), to_f32(p.v[w + 1]), to_f32(p.v[w + 2]), to_f32(p.v[w + 3]), r);
  *reinterpret_cast<Pack<uint32_t, W / 4>*>(q) = o;
}

// LPR lanes (a wave or the workgroup) a row, up to NV 16-byte pieces of it a lane, held in
// registers between the maximum and the codes; NV == 0: rows of any length, read twice.
template <typename T, int LPR, int NV>
__global__ void __launch_bounds__(QTHREADS)
int8_quantize_kernel(const T* __restrict__ x, int64_t rows, int64_t cols, int64_t ldx, int vec,
                     int8_t* __restrict__ q, int64_t ldq, float* __restrict__ scales) {
  constexpr int W = 16 / (int)sizeof(T), PER = QTHREADS / LPR;
  __shared__ uint32_t wave_max[2][QTHREADS / 64];
  const int l = threadIdx.x % LPR;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * PER; r0 < rows; r0 += (int64_t)gridDim.x * PER, turn ^= 1) {
    const int64_t row = r0 + threadIdx.x / LPR;
    const bool in = row < rows;
    const T* const from = x + (in ? row : 0) * ldx;
    uint32_t m = 0;
    Pack<T, W> p[NV > 0 ? NV : 1];
    if constexpr (NV > 0) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int64_t at = (int64_t)(v * LPR + l) * W;
        if (in && at < cols) {
          p[v] = load_pack<T, W>(from, at, vec != 0);
        } else {
#pragma unroll
          for (int w = 0; w < W; ++w) p[v].v[w] = from_f32<T>(0.0f);
        }
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) m = pack_amax<T, W>(p[v], m);
    } else {
      for (int64_t at = (int64_t)l * W; in && at < cols; at += LPR * W)
        m = pack_amax<T, W>(load_pack<T, W>(from, at, vec != 0), m);
    }
    m = reduce_u32<64>(m, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    if constexpr (LPR == QTHREADS) {
      // (two rows' maxima side by side: one barrier a row)
      if ((threadIdx.x & 63) == 0) wave_max[turn][threadIdx.x >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < QTHREADS / 64; ++w) m = max(m, wave_max[turn][w]);
    }
    const RowScale s = row_scale(m);
    if (!in) continue;
    if (l == 0) scales[row] = s.scale;
    int8_t* const to = q + row * ldq;
    if constexpr (NV > 0) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int64_t at = (int64_t)(v * LPR + l) * W;
        if (at < cols) store_codes<T, W>(p[v], s, to + at);
      }
    } else {
      for (int64_t at = (int64_t)l * W; at < cols; at += LPR * W)
        store_codes<T, W>(load_pack<T, W>(from, at, vec != 0), s, to + at);
    }
  }
}

template <typename T>
using QuantFn = void (*)(const T*, int64_t, int64_t, int64_t, int, int8_t*, int64_t, float*);
template <typename T>
QuantFn<T> quant_pick(int64_t cols, int* rows_per_group) {
  constexpr int W = 16 / (int)sizeof(T);
  *rows_per_group = 4;
  if (cols <= 64 * W) return int8_quantize_kernel<T, 64, 1>;
  if (cols <= 64 * 4 * W) return int8_quantize_kernel<T, 64, 4>;
  *rows_per_group = 1;
  if (cols <= 256 * 4 * W) return int8_quantize_kernel<T, 256, 4>;
  if (cols <= 256 * 8 * W) return int8_quantize_kernel<T, 256, 8>;
  return int8_quantize_kernel<T, 256, 0>;
}
template <typename T>
hipError_t quant_launch(const void* x, int64_t rows, int64_t cols, int64_t ldx, int8_t* q, int64_t ldq,
                        float* scales, hipStream_t stream) {
  int per;
  const QuantFn<T> fn = quant_pick<T>(cols, &per);
  const int vec = (uintptr_t)x % 16 == 0 && ldx * (int64_t)sizeof(T) % 16 == 0;
  const int64_t groups = (rows + per - 1) / per;
  const int64_t grid = groups < (1 << 20) ? groups : (1 << 20);
  fn<<<dim3((unsigned)grid), dim3(QTHREADS), 0, stream>>>((const T*)x, rows, cols, ldx, vec, q, ldq, scales);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// The product, simplest form: 128x128 tiles, four waves of 64x64, 64 bytes of K a step
// through registers into one LDS stage.
constexpr int BT = 128, BKS = 64, LDR = BKS + 16;      // (16 bytes of padding a row)

__global__ void __launch_bounds__(256)
int8_simple_kernel(Int8Args a) {
  __shared__ __attribute__((aligned(16))) int8_t la[BT * LDR], lb[BT * LDR];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t row0 = (int64_t)blockIdx.y * BT, first = 0, end = a.rows;
  int g = 0;
  if (a.mode == MODE_CONTIGUOUS) {
    int64_t block = blockIdx.y;
    for (g = 0; g < a.G; ++g) {
      row0 = min(max((int64_t)a.group[g], (int64_t)0), a.rows);
      end = min(max((int64_t)a.group[g + 1], row0), a.rows);
      const int64_t n = (end - row0 + BT - 1) / BT;
      if (block < n) break;
      block -= n;
    }
    if (g == a.G) return;
    row0 += block * BT;
  } else if (a.mode == MODE_MASKED) {
    g = blockIdx.z;
    first = (int64_t)g * a.rows;
    end = min((int64_t)a.group[g], a.rows);
  }
  if (row0 >= end) return;
  const int mv = (int)min((int64_t)BT, end - row0);
  const int64_t n0 = (int64_t)blockIdx.x * BT;
  const int nv = (int)min((int64_t)BT, a.N - n0);
  const int8_t* const pa = a.a + (first + row0) * a.K;
  const int8_t* const pb = a.b + ((int64_t)g * a.N + n0) * a.K;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  v16i acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = v16i{};
  for (int64_t k0 = 0; k0 < a.K; k0 += BKS) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int i = c * 256 + threadIdx.x, r = i >> 2, ch = (i & 3) * 16;
      u32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
      if (k0 + ch < a.K) {
        if (r < mv) x = *reinterpret_cast<const u32x4*>(pa + r * a.K + k0 + ch);
        if (r < nv) y = *reinterpret_cast<const u32x4*>(pb + r * a.K + k0 + ch);
      }
      *reinterpret_cast<u32x4*>(la + r * LDR + ch) = x;
      *reinterpret_cast<u32x4*>(lb + r * LDR + ch) = y;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4i fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = *reinterpret_cast<const v4i*>(la + (wm + i * 32 + (lane & 31)) * LDR + h * 32 + (lane >> 5) * 16);
        fb[i] = *reinterpret_cast<const v4i*>(lb + (wn + i * 32 + (lane & 31)) * LDR + h * 32 + (lane >> 5) * 16);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
    __syncthreads();
  }
  // (b is the first operand: lane l holds row l % 32 of a's fragment and columns 8 t + 4 (l / 32) + e of b's)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = wm + i * 32 + (lane & 31);
    if (r >= mv) continue;
    const float s = a.sa[first + row0 + r];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int c = wn + j * 32 + t * 8 + (lane >> 5) * 4;
        if (c >= nv) continue;
        const float* const sb = a.sb + (int64_t)g * a.N + n0 + c;
        Pack<bf16_t, 4> o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o.v[e] = (bf16_t)((float)acc[i][j][4 * t + e] * s * sb[e]);
        *reinterpret_cast<Pack<bf16_t, 4>*>(a.d + (first + row0 + r) * a.N + n0 + c) = o;
      }
  }
}

}  // namespace

hipError_t launch_int8_quantize(const void* x, int type, int64_t rows, int64_t cols, int64_t ldx, int8_t* q,
                                int64_t ldq, float* scales, hipStream_t stream) {
  if (type == TYPE_F32) return quant_launch<float>(x, rows, cols, ldx, q, ldq, scales, stream);
  if (type == TYPE_BF16) return quant_launch<bf16_t>(x, rows, cols, ldx, q, ldq, scales, stream);
  return quant_launch<f16_t>(x, rows, cols, ldx, q, ldq, scales, stream);
}

hipError_t launch_int8(const Int8Args& args, const DeviceInfo& dev, int expected_m, hipStream_t stream) {
  const dim3 grid((unsigned)((args.N + BT - 1) / BT), (unsigned)((args.rows + BT - 1) / BT + (args.mode == MODE_CONTIGUOUS ? args.G : 0)),
                  args.mode == MODE_MASKED ? (unsigned)args.G : 1);
  int8_simple_kernel<<<grid, dim3(256), 0, stream>>>(args);
  return hipGetLastError();
}

void int8_kernels(std::vector<const void*>& out) {
  int per;
  for (int64_t cols : {16, 1024, 2048, 8192, 16384, 32768}) {
    out.push_back((const void*)quant_pick<float>(cols, &per));
    out.push_back((const void*)quant_pick<bf16_t>(cols, &per));
    out.push_back((const void*)quant_pick<f16_t>(cols, &per));
  }
  out.push_back((const void*)int8_simple_kernel);
}

}  // namespace fp8g
