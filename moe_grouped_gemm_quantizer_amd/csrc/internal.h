// Internal declarations shared by the HIP translation units of libfp8gemm.
// Nothing here is part of the C ABI (include/fp8gemm.h is).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <vector>
#include <stdint.h>

namespace fp8g {

// Per-device facts the launchers need, queried once per device.
struct DeviceInfo {
  int ok;          // 1 when the device is a usable gfx950
  int cu_count;    // compute units (256 on MI355X)
};
// Fills *info for the current device; returns 0 on success.
int current_device_info(DeviceInfo* info);

// Launchers (arguments already validated by the C entry points). The
// quantiser takes fp32 (T = float) or bf16 bit patterns (T = uint16_t).
template <typename T>
hipError_t launch_quantize(const T* x, int64_t rows, int64_t cols, int64_t ldx,
                           int block_rows, uint8_t* q, int64_t ldq, float* scales,
                           int64_t s_stride_row, int64_t s_stride_col, hipStream_t stream,
                           int cu_count);

// MODE_PERTENSOR: one scale per operand (sa, sb point at one float each);
// the MFMA accumulates over all of K and the epilogue applies sa * sb once.
// Per-tensor quantisation: one scale (written to *scale) for the whole matrix.
hipError_t launch_quantize_tensor(const float* x, int64_t rows, int64_t cols, int64_t ldx,
                                  uint8_t* q, int64_t ldq, float* scale, hipStream_t stream);

enum GemmMode { MODE_DENSE = 0, MODE_CONTIGUOUS = 1, MODE_MASKED = 2, MODE_PERTENSOR = 3 };

struct GemmArgs {
  const uint8_t* a;        // e4m3 rows, K contiguous
  const float* sa;         // [K/128][sa_ld]
  const uint8_t* b;        // e4m3 [G][N][K]
  const float* sb;         // [G][N/128][K/128]
  uint16_t* d;             // bf16 bits, rows of N
  const int32_t* group;    // contiguous: offsets [G+1]; masked: counts [G]; dense: null
  int64_t rows;            // dense: M; contiguous: M_total; masked: max_m
  int64_t sa_ld;           // row count of the sa layout (M, M_total or G*max_m)
  int64_t N;
  int64_t K;
  int G;
  int mode;
  // Set by the launcher only (the entry points leave the defaults):
  int split_base = 0;      // contiguous, splits > 1: tiles from here on run as K pieces
  int splits = 1;          // contiguous: K pieces per tile past split_base (1: none)
  float* ws = nullptr;     // split workspace: fp32 partial tiles [piece][BM][BN]
  struct SplitMeta* ws_meta = nullptr;  // split workspace: what the reduction reads
  // Dense only, set by the fused entry point: the bf16 result is also
  // quantised per 1x128 block into qd [rows][N] (e4m3) with scales
  // sd [N/128][rows]; d may then be null (no bf16 output).
  uint8_t* qd = nullptr;
  float* sd = nullptr;
  // Per-tensor only: operand formats, fmt_a | fmt_b << 4 (Fp8Format codes).
  int fmts = 0;
};

// Written by the GEMM kernel for the reduction of its split tail: the
// number of tail tiles (0: nothing to reduce), the pieces per tile, and
// where each tail tile's output goes. SplitTile records follow the header.
struct SplitTile {
  int64_t d_off;           // offset of the tile's first output element in d
  int mvalid, nvalid;      // rows and columns of the tile that exist
};
struct SplitMeta {
  int tail;
  int splits;
  int pad[2];
};
// Launch of a validated GEMM call. ws/ws_bytes: caller-owned workspace for a
// contiguous call's split tail (null/0: the call runs unsplit; a workspace
// smaller than contiguous_workspace_bytes is not used).
hipError_t launch_gemm(const GemmArgs& args, const DeviceInfo& dev, int expected_m, void* ws,
                       size_t ws_bytes, hipStream_t stream);
// Workspace a contiguous call with these sizes can use (0: it never splits).
size_t contiguous_workspace_bytes(const GemmArgs& args, const DeviceInfo& dev);

// FP8 element formats (the MFMA's operand format codes).
enum Fp8Format { FMT_E4M3 = 0, FMT_E5M2 = 1 };

// Delayed-scaling quantiser (quantize.hip): scale from the amax window,
// codes in format fmt, this step's amax into history[slot].
hipError_t launch_quantize_delayed(const float* x, int64_t rows, int64_t cols, int64_t ldx,
                                   int fmt, float* history, int hist_len, int slot, uint8_t* q,
                                   int64_t ldq, float* scale, hipStream_t stream);

// Kernel table (gemm.hip): the text naming the kernel a GEMM call of these
// arguments launches (snprintf's return value), and the process-wide switch
// between the shape-specialised instantiations and the generic ones (on by
// default; both give the same bits).
int describe_gemm(const GemmArgs& args, int expected_m, char* buf, size_t len);
void set_shape_specialisation(int enable);
// Every kernel of the library (for warm-up: loading each one's code object
// onto the current device ahead of the first call).
void gemm_kernels(std::vector<const void*>& out);
void quantize_kernels(std::vector<const void*>& out);

// Element types of inputs that are not 8-bit codes (FP8G_TYPE_*).
enum ElemType { TYPE_F32 = 0, TYPE_BF16 = 1, TYPE_F16 = 2 };

// Routing (route.hip); arguments as for moe_route and moe_route_backward.
struct RouteCall {
  const void* logits;
  int type;
  int64_t T, ld, max_m;
  int E, k, renorm, align;
  float coef;
  const uint8_t* mask;
  int32_t *ids, *counts, *routed, *offsets, *slots;
  float *weights, *prob_sum, *loss;
  void* workspace;
};
struct RouteBwdCall {
  const void* logits;
  int type;
  int64_t T, ld, ldd;
  int E, k, renorm;
  float coef;
  const int32_t *ids, *counts, *routed;
  const float *dw, *dloss;
  void* d_logits;
};
size_t route_workspace_bytes(int64_t T, int E);
hipError_t launch_route(const RouteCall& c, hipStream_t stream);
hipError_t launch_route_backward(const RouteBwdCall& c, hipStream_t stream, int cu_count);
// What follows the rows' kernel of more than one block, or of none: the scan of the blocks' counts,
// slots, offsets and loss (a choice's rank inside its block is in its slot by then).
hipError_t launch_route_places(const RouteCall& c, hipStream_t stream);
void route_kernels(std::vector<const void*>& out);
// Routing by scores (route_scored.hip); arguments as for moe_route_scored and its gradient.
enum RouteScore { SCORE_SIGMOID = 0, SCORE_SOFTMAX = 1 };
struct ScoredCall {
  RouteCall route;
  const float* bias;
  int score, groups, open, best;
  float scale;
};
struct ScoredBwdCall {
  RouteBwdCall route;
  int score;
  float scale;
};
hipError_t launch_route_scored(const ScoredCall& c, hipStream_t stream, int cu_count);
hipError_t launch_route_scored_backward(const ScoredBwdCall& c, hipStream_t stream, int cu_count);
void route_scored_kernels(std::vector<const void*>& out);

// The weight gradient (wgrad.hip).
hipError_t launch_quantize_transpose(const void* x, int type, int64_t rows, int64_t cols,
                                     int64_t ldx, int fmt, uint8_t* qt, int64_t ldq, uint8_t* st,
                                     hipStream_t stream);
struct WgradArgs {
  const uint8_t *a, *sa, *b, *sb;      // codes [M][lda], [N][ldb]; exponent bytes [T/128][M], [T/128][N]
  uint16_t* d;                         // bf16 bits [G][M][N]
  const int32_t* group;                // offsets [G + 1], or null (one expert, all T tokens)
  int64_t lda, ldb, T, M, N;
  int G;
};
hipError_t launch_wgrad(const WgradArgs& args, int fmt_a, int fmt_b, const DeviceInfo& dev,
                        hipStream_t stream);
void wgrad_kernels(std::vector<const void*>& out);

// Gradient norm and clipping (clip.hip).
size_t grad_norm_workspace_bytes(const int64_t* numels, int n);
hipError_t launch_grad_norm_sq(const void* const* grads, const int64_t* numels, const int* types,
                               int n, double* sumsq, void* workspace, hipStream_t stream);
hipError_t launch_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels,
                            const int* types, int n, const double* sumsq, float max_norm,
                            float* norm, hipStream_t stream);
void clip_kernels(std::vector<const void*>& out);

// Products in 8-bit integers (int8.hip).
hipError_t launch_int8_quantize(const void* x, int type, int64_t rows, int64_t cols, int64_t ldx, int8_t* q,
                                int64_t ldq, float* scales, hipStream_t stream);
struct Int8Args {
  const int8_t* a;         // codes, rows of K
  const float* sa;         // a scale for each row of a
  const int8_t* b;         // codes [G][N][K]
  const float* sb;         // [G][N]
  uint16_t* d;             // bf16 bits, rows of N
  const int32_t* group;    // contiguous: offsets [G + 1]; masked: counts [G]; dense: null
  int64_t rows;            // dense: M; contiguous: M_total; masked: max_m
  int64_t N, K;
  int G, mode;             // MODE_DENSE, MODE_CONTIGUOUS or MODE_MASKED
  int round = 0;           // set by the launcher: workgroups of a round
};
hipError_t launch_int8(const Int8Args& args, const DeviceInfo& dev, int expected_m, hipStream_t stream);
void int8_kernels(std::vector<const void*>& out);

// The AdamW step (adamw.hip); arguments as for adamw_step.
struct AdamwCall {
  void* const* params;
  const int* param_types;
  const void* const* grads;
  const int* grad_types;
  void* const* m;
  void* const* v;
  uint8_t* const* ms;      // null: states in 32 bits
  uint8_t* const* vs;
  void* const* copies;     // null: none
  const int* copy_types;
  const int64_t* numels;
  int n;
  const int64_t* step_at;
  int64_t step;
  const float* lr_at;
  double lr, beta1, beta2, eps, weight_decay;
  const double* sumsq;
  float max_norm;
  float* norm;
  uint32_t seed;
  const void* table;       // null, or what adamw_table_fill wrote, in device memory
};
hipError_t launch_adamw(const AdamwCall& c, hipStream_t stream);
size_t adamw_table_bytes(int n);
bool adamw_table_fill(const AdamwCall& c, void* table);  // (false: too many chunks for a table)
void adamw_kernels(std::vector<const void*>& out);

// The allocation-free contiguous entry point's scratch: its size, and its
// device address on `device` (looked up once per device; nullptr on failure;
// call with that device current).
size_t noalloc_scratch_bytes();
void* scratch_ptr(int device);

}  // namespace fp8g
