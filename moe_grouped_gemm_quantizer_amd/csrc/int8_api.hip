// C entry points of the products in 8-bit integers: argument validation and launch. As in
// fp8gemm_api.hip, every check comes before the first HIP call.

#include <stddef.h>

#include "../../include/fp8gemm.h"
#include "internal.h"

using namespace fp8g;

namespace {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
constexpr int64_t kMaxK = (1 << 17) - 16;             // K 2^14 < 2^31: the sum fits 32 bits
constexpr int64_t kMaxRows = int64_t(1) << 30;
inline fp8g_status launched(hipError_t e) { return e == hipSuccess ? FP8G_OK : FP8G_ERR_LAUNCH; }

fp8g_status check_nk(int64_t N, int64_t K) {
  if (N <= 0 || K <= 0 || N % 16 != 0 || K % 16 != 0) return FP8G_ERR_SHAPE;
  if (K > kMaxK || N > (int64_t(1) << 27)) return FP8G_ERR_UNSUPPORTED;
  return FP8G_OK;
}

fp8g_status check_ptrs(const Int8Args& a) {
  if (!a.a || !a.sa || !a.b || !a.sb || !a.d) return FP8G_ERR_NULL_PTR;
  if (a.mode != MODE_DENSE && !a.group) return FP8G_ERR_NULL_PTR;
  if (!aligned(a.a, 16) || !aligned(a.b, 16) || !aligned(a.d, 16) || !aligned(a.sa, 4) ||
      !aligned(a.sb, 4) || !aligned(a.group, 4))
    return FP8G_ERR_ALIGN;
  return FP8G_OK;
}

// Tiles of 128x128 for row blocks `mb`, over all experts. A launch holds fewer than 2^32 threads, 256 a tile.
constexpr int64_t kMaxTiles = (1 << 24) - 1;
bool too_many_tiles(int64_t mb, int64_t N, int64_t G) {
  const int64_t nb = (N + 127) / 128;
  return mb > kMaxTiles / nb || G > kMaxTiles / (mb * nb > 0 ? mb * nb : 1);
}

fp8g_status run(const Int8Args& a, int expected_m, hipStream_t stream) {
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  return launched(launch_int8(a, dev, expected_m, stream));
}

}  // namespace

extern "C" {

fp8g_status int8_quantize(const void* x, int type, int64_t rows, int64_t cols, int64_t ldx, int8_t* q,
                          int64_t ldq, float* scales, hipStream_t stream) {
  if (rows < 0 || cols <= 0 || cols % 16 != 0) return FP8G_ERR_SHAPE;
  if (type < FP8G_TYPE_F32 || type > FP8G_TYPE_F16) return FP8G_ERR_UNSUPPORTED;
  if (rows == 0) return FP8G_OK;
  if (!x || !q || !scales) return FP8G_ERR_NULL_PTR;
  if (ldx < cols || ldq < cols) return FP8G_ERR_STRIDE;
  if (!aligned(x, type == FP8G_TYPE_F32 ? 4 : 2) || !aligned(q, 16) || ldq % 16 != 0 || !aligned(scales, 4))
    return FP8G_ERR_ALIGN;
  DeviceInfo dev;
  if (current_device_info(&dev) != 0) return FP8G_ERR_DEVICE;
  return launched(launch_int8_quantize(x, type, rows, cols, ldx, q, ldq, scales, stream));
}

fp8g_status gemm_int8(const int8_t* a, const float* sa, const int8_t* b, const float* sb, uint16_t* d,
                      int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  if (M < 0) return FP8G_ERR_SHAPE;
  const fp8g_status s = check_nk(N, K);
  if (s != FP8G_OK) return s;
  if (M == 0) return FP8G_OK;
  const Int8Args args{a, sa, b, sb, d, nullptr, M, N, K, 1, MODE_DENSE};
  const fp8g_status p = check_ptrs(args);
  if (p != FP8G_OK) return p;
  if (M > kMaxRows || too_many_tiles((M + 127) / 128, N, 1)) return FP8G_ERR_UNSUPPORTED;
  return run(args, 0, stream);
}

fp8g_status grouped_gemm_int8_contiguous(const int8_t* a, const float* sa, const int8_t* b, const float* sb,
                                         uint16_t* d, const int32_t* group_offsets, int G, int64_t M_total,
                                         int64_t N, int64_t K, hipStream_t stream) {
  if (G < 0 || M_total < 0) return FP8G_ERR_SHAPE;
  const fp8g_status s = check_nk(N, K);
  if (s != FP8G_OK) return s;
  if (G == 0 || M_total == 0) return FP8G_OK;
  const Int8Args args{a, sa, b, sb, d, group_offsets, M_total, N, K, G, MODE_CONTIGUOUS};
  const fp8g_status p = check_ptrs(args);
  if (p != FP8G_OK) return p;
  // (every expert may end inside a row block)
  if (G > 1024 || M_total > kMaxRows || too_many_tiles((M_total + 127) / 128 + G, N, 1))
    return FP8G_ERR_UNSUPPORTED;
  return run(args, 0, stream);
}

fp8g_status grouped_gemm_int8_masked(const int8_t* a, const float* sa, const int8_t* b, const float* sb,
                                     uint16_t* d, const int32_t* masked_m, int G, int64_t max_m, int64_t N,
                                     int64_t K, int expected_m, hipStream_t stream) {
  if (G < 0 || max_m < 0) return FP8G_ERR_SHAPE;
  const fp8g_status s = check_nk(N, K);
  if (s != FP8G_OK) return s;
  if (G == 0 || max_m == 0) return FP8G_OK;
  const Int8Args args{a, sa, b, sb, d, masked_m, max_m, N, K, G, MODE_MASKED};
  const fp8g_status p = check_ptrs(args);
  if (p != FP8G_OK) return p;
  if (G > 1024 || max_m > kMaxRows || too_many_tiles((max_m + 127) / 128, N, G)) return FP8G_ERR_UNSUPPORTED;
  return run(args, expected_m, stream);
}

}  // extern "C"
