// Global gradient norm and clipping over a list of tensors.
//
// norm = sqrt(sum over all tensors of x^2); each gradient is multiplied by
// min(1, max_norm / (norm + 1e-6)). Both passes are HBM streams. Squares are
// formed and added in fp64: an fp32 square overflows from 1.8e19 on and
// vanishes below 1e-23, and the vector unit's fp64 rate (one fma per lane
// and cycle as in fp32) is far above what HBM feeds it.
//
// Measured: 8 x 29.4M bf16 (470 MB read, then read and written): norm 77-81 us
// (6 TB/s), clipping 141-148 us (6.4 TB/s); 300 tensors of 50M values, half of
// them fp32: 43 + 68 us in three launches each, less than the host takes to
// list them; 12 tensors of 40,000 values 5.1 + 4.5 us.
//
// The list travels in the kernel's arguments, up to 112 tensors a launch
// (4 KB of arguments): nothing of it stays on the device or in the library.

#include <vector>

#include "elem.h"
#include "internal.h"

namespace fp8g {
namespace {

using namespace elem;

constexpr int THREADS = 256;
constexpr int MAX_T = 112;                             // tensors of a launch
// Elements of a chunk: small ones where the list would otherwise leave CUs without
// work, large ones where there is plenty (each chunk costs a search in the table).
constexpr int64_t CHUNK_MIN = 8192, CHUNK_MAX = 32768;
// A list of up to TINY chunks of CHUNK_TINY values is summed by one workgroup,
// two chunks a wave: one launch instead of two, which is what such a call costs
// (two launches against one: 1 tensor of 16,384 values, 8 chunks, 4.7 / 3.0 us; 12 tensors,
// 40,000 values, 30 chunks 5.0 / 4.4; 32 tensors 4.9 / 4.5; 40 chunks 5.1 / 5.3 to 6.5; one tensor of
// 131,072 values, 64 chunks, 4.9 / 6.7; 100 small tensors 5.0 / 9.7).
constexpr int64_t TINY = 32, CHUNK_TINY = 2048;
constexpr int64_t MAX_GRID = 2048;                     // eight workgroups per CU
constexpr int64_t STREAM_BYTES = 192 << 20;            // lists from here on outgrow the caches

struct Table {
  const void* x[MAX_T];
  void* y[MAX_T];
  int64_t numel[MAX_T];
  int end[MAX_T];                                      // chunks of this tensor and those before it
  uint8_t type[MAX_T];
  int n, chunk;
};

int64_t chunks_of(int64_t numel, int64_t chunk) { return (numel + chunk - 1) / chunk; }

// A list's chunk in the norm: the large one from twice a full grid of them on.
int64_t chunk_for(const int64_t* numels, int n) {
  int64_t total = 0, tiny = 0;
  for (int i = 0; i < n && total < 2 * MAX_GRID * CHUNK_MAX; ++i) {
    total += numels[i];
    tiny += chunks_of(numels[i], CHUNK_TINY);
  }
  if (tiny <= TINY) return CHUNK_TINY;                 // (so at most TINY tensors that are not empty)
  return total < 2 * MAX_GRID * CHUNK_MAX ? CHUNK_MIN : CHUNK_MAX;
}

// And in the clipping, where a short list takes the smallest chunks on as many CUs (chunks
// of 8192 / 2048: 131,072 values in 1 tensor 3.8 / 2.9 us, in 12 4.0 / 3.1; 1M values in 1
// 4.0 / 3.3, in 100 4.6 / 4.0).
constexpr int64_t CLIP_SHORT = 1 << 20;
int64_t clip_chunk_for(const int64_t* numels, int n) {
  int64_t total = 0;
  for (int i = 0; i < n && total <= CLIP_SHORT; ++i) total += numels[i];
  return total <= CLIP_SHORT ? CHUNK_TINY : chunk_for(numels, n);
}

// The tensor of chunk c and the chunk's place in it.
__device__ __forceinline__ int find(const Table& t, int c, int64_t& at) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (c < t.end[mid]) hi = mid;
    else lo = mid + 1;
  }
  at = (int64_t)(c - (lo ? t.end[lo - 1] : 0)) * t.chunk;
  return lo;
}

// (by NT threads, of which this is number t)
template <int NT, typename T>
__device__ __forceinline__ double chunk_sum(const T* __restrict__ x, int n, int t) {
  constexpr int W = 16 / (int)sizeof(T);
  double s = 0.0;
  int done = 0;
  if ((uintptr_t)x % 16 == 0) {
    const int packs = n / W;
    done = packs * W;
#pragma unroll 4
    for (int i = t; i < packs; i += NT) {
      const Pack<T, W> p = reinterpret_cast<const Pack<T, W>*>(x)[i];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const double v = (double)to_f32(p.v[w]);
        s = __builtin_fma(v, v, s);
      }
    }
  }
  for (int i = done + t; i < n; i += NT) {
    const double v = (double)to_f32(x[i]);
    s = __builtin_fma(v, v, s);
  }
  return s;
}

template <int NT>
__device__ __forceinline__ double table_chunk_sum(const Table& table, int c, int t) {
  int64_t at;
  const int i = find(table, c, at);
  const int64_t left = table.numel[i] - at;
  const int n = (int)(left < table.chunk ? left : table.chunk);
  if (table.type[i] == TYPE_F32) return chunk_sum<NT>((const float*)table.x[i] + at, n, t);
  if (table.type[i] == TYPE_BF16) return chunk_sum<NT>((const bf16_t*)table.x[i] + at, n, t);
  return chunk_sum<NT>((const f16_t*)table.x[i] + at, n, t);
}

// Sum over the workgroup, in lane and wave order.
template <int NT>
__device__ __forceinline__ double group_sum(double s, double* lds) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < NT / 64; w += 4) s += (lds[w] + lds[w + 1]) + (lds[w + 2] + lds[w + 3]);
  return s;
}

// Chunks blockIdx.x, + gridDim.x, ...: one partial sum per workgroup.
__global__ void __launch_bounds__(THREADS)
norm_partial_kernel(Table t, double* __restrict__ part) {
  __shared__ double lds[THREADS / 64];
  double s = 0.0;
  const int chunks = t.end[t.n - 1];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) s += table_chunk_sum<THREADS>(t, c, threadIdx.x);
  s = group_sum<THREADS>(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

constexpr int TINY_THREADS = 1024;
__global__ void __launch_bounds__(TINY_THREADS)
norm_tiny_kernel(Table t, double* __restrict__ sumsq) {
  __shared__ double lds[TINY_THREADS / 64];
  double s = 0.0;
  const int chunks = t.end[t.n - 1];
  for (int c = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); c < chunks; c += TINY_THREADS / 64)
    s += table_chunk_sum<64>(t, c, threadIdx.x & 63);
  s = group_sum<TINY_THREADS>(s, lds);
  if (threadIdx.x == 0) *sumsq = s;
}

__global__ void __launch_bounds__(THREADS)
norm_finish_kernel(const double* __restrict__ part, int n, double* __restrict__ sumsq) {
  __shared__ double lds[THREADS / 64];
  double s = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < n; i += THREADS) s += part[i];
  s = group_sum<THREADS>(s, lds);
  if (threadIdx.x == 0) *sumsq = s;
}

// The product rounded to fp32, then to the type. (Left to itself the compiler
// turns some fp16 products into a mixed-precision fma, which rounds once, so
// that an element's result would depend on the path it takes.) A factor below
// fp32's normal numbers comes as fp64: in fp32 it would lose bits, or vanish, where
// gradients near the end of the range still have normal products.
template <typename T, typename F>
__device__ __forceinline__ T scaled(T x, F f) {
  float p = (float)((F)to_f32(x) * f);
  asm("" : "+v"(p));
  return from_f32<T>(p);
}

// Stores are non-temporal: the next reader is another kernel, and the list's
// own values are what should stay in the caches (8 x 29M bf16, norm and
// clipping: 278 -> 246 us; 8 x 2M: 22.6 -> 22.4). STREAM: so are the loads,
// for a list larger than the caches, where they would push out what the
// norm's pass left there (8 x 29M: 246 -> 233 us, 8 x 16M: 135 -> 131; but
// 8 x 8M 66.5 -> 69, 8 x 2M 22.4 -> 29).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <bool STREAM, typename T, typename F>
__device__ __forceinline__ void chunk_scale(const T* x, T* y, int n, F f) {
  constexpr int W = 16 / (int)sizeof(T);
  int done = 0;
  if (((uintptr_t)x | (uintptr_t)y) % 16 == 0) {
    const int packs = n / W;
    done = packs * W;
#pragma unroll 4
    for (int i = threadIdx.x; i < packs; i += THREADS) {
      const u32x4* const at = reinterpret_cast<const u32x4*>(x) + i;
      Pack<T, W> p = __builtin_bit_cast(Pack<T, W>, STREAM ? __builtin_nontemporal_load(at) : *at);
#pragma unroll
      for (int w = 0; w < W; ++w) p.v[w] = scaled(p.v[w], f);
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4, p), reinterpret_cast<u32x4*>(y) + i);
    }
  }
  for (int i = done + threadIdx.x; i < n; i += THREADS) y[i] = scaled(x[i], f);
}

template <bool STREAM, typename F>
__device__ __forceinline__ void table_chunk_scale(const Table& t, int i, int64_t at, F f) {
  const int64_t left = t.numel[i] - at;
  const int n = (int)(left < t.chunk ? left : t.chunk);
  if (t.type[i] == TYPE_F32)
    chunk_scale<STREAM>((const float*)t.x[i] + at, (float*)t.y[i] + at, n, f);
  else if (t.type[i] == TYPE_BF16)
    chunk_scale<STREAM>((const bf16_t*)t.x[i] + at, (bf16_t*)t.y[i] + at, n, f);
  else
    chunk_scale<STREAM>((const f16_t*)t.x[i] + at, (f16_t*)t.y[i] + at, n, f);
}

// (n == 0: one workgroup writes the norm)
template <bool STREAM>
__global__ void __launch_bounds__(THREADS)
clip_kernel(Table t, const double* __restrict__ sumsq, float max_norm, float* __restrict__ norm,
            int write_norm) {
  const double nrm = sqrt(*sumsq);
  if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)nrm;
  const double q = (double)max_norm / (nrm + 1e-6);
  const float f = q >= 1.0 ? 1.0f : (float)q;          // (NaN stays NaN)
  const int chunks = t.n ? t.end[t.n - 1] : 0;
  // (last chunks first: of what the norm's pass read, the end is what the
  // caches still hold)
  for (int c = chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    int64_t at;
    const int i = find(t, c, at);
    if (t.x[i] == t.y[i] && f == 1.0f) continue;
    if (q < 0x1p-126) table_chunk_scale<STREAM>(t, i, at, q);
    else table_chunk_scale<STREAM>(t, i, at, f);
  }
}

// The next tensors of the list that fit a launch; empty ones are left out.
// Returns the launch's grid, 0 when the list is done.
int64_t fill(Table& t, int& i, const void* const* xs, void* const* ys, const int64_t* numels,
             const int* types, int n) {
  t.n = 0;
  int64_t chunks = 0;
  for (; i < n && t.n < MAX_T; ++i) {
    if (numels[i] == 0) continue;
    const int64_t c = chunks_of(numels[i], t.chunk);
    if (chunks + c > 0x7FFFFFFF) break;                // (each tensor fits by itself: checked before)
    chunks += c;
    t.x[t.n] = xs[i];
    t.y[t.n] = ys ? ys[i] : nullptr;
    t.numel[t.n] = numels[i];
    t.type[t.n] = (uint8_t)types[i];
    t.end[t.n] = (int)chunks;
    ++t.n;
  }
  return chunks < MAX_GRID ? chunks : MAX_GRID;
}

}  // namespace

// One fp64 partial sum per workgroup of every launch: a launch has at most
// MAX_GRID of them, and at most one per chunk.
size_t grad_norm_workspace_bytes(const int64_t* numels, int n) {
  const int64_t chunk = chunk_for(numels, n);
  int64_t parts = 0, chunks = 0;
  int tensors = 0;
  for (int i = 0; i < n; ++i) {
    if (numels[i] == 0) continue;
    const int64_t c = chunks_of(numels[i], chunk);
    if (tensors == MAX_T || chunks + c > 0x7FFFFFFF) {
      parts += chunks < MAX_GRID ? chunks : MAX_GRID;
      chunks = 0;
      tensors = 0;
    }
    chunks += c;
    ++tensors;
  }
  parts += chunks < MAX_GRID ? chunks : MAX_GRID;
  return (size_t)parts * sizeof(double);
}

hipError_t launch_grad_norm_sq(const void* const* grads, const int64_t* numels, const int* types,
                               int n, double* sumsq, void* workspace, hipStream_t stream) {
  Table t;
  t.chunk = (int)chunk_for(numels, n);
  double* part = (double*)workspace;
  int parts = 0, i = 0;
  for (;;) {
    const int64_t grid = fill(t, i, grads, nullptr, numels, types, n);
    if (grid == 0) break;
    if (t.chunk == CHUNK_TINY) {                       // (such a list fits one table)
      norm_tiny_kernel<<<dim3(1), dim3(TINY_THREADS), 0, stream>>>(t, sumsq);
      return hipGetLastError();
    }
    norm_partial_kernel<<<dim3((unsigned)grid), dim3(THREADS), 0, stream>>>(t, part + parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;                     // (the sum would be of what is not there)
    parts += (int)grid;
  }
  norm_finish_kernel<<<dim3(1), dim3(THREADS), 0, stream>>>(part, parts, sumsq);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels,
                            const int* types, int n, const double* sumsq, float max_norm,
                            float* norm, hipStream_t stream) {
  Table t;
  t.chunk = (int)clip_chunk_for(numels, n);
  int64_t bytes = 0;
  for (int j = 0; j < n && bytes < STREAM_BYTES; ++j) bytes += numels[j] * (types[j] == TYPE_F32 ? 4 : 2);
  const auto kernel = bytes >= STREAM_BYTES ? clip_kernel<true> : clip_kernel<false>;
  int i = 0, first = 1;
  for (;;) {
    const int64_t grid = fill(t, i, grads, outs, numels, types, n);
    if (grid == 0 && !first) break;
    kernel<<<dim3((unsigned)(grid ? grid : 1)), dim3(THREADS), 0, stream>>>(t, sumsq, max_norm, norm,
                                                                            first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    first = 0;
    if (grid == 0) break;
  }
  return hipSuccess;
}

void clip_kernels(std::vector<const void*>& out) {
  out.push_back((const void*)norm_partial_kernel);
  out.push_back((const void*)norm_tiny_kernel);
  out.push_back((const void*)norm_finish_kernel);
  out.push_back((const void*)clip_kernel<false>);
  out.push_back((const void*)clip_kernel<true>);
}

}  // namespace fp8g
