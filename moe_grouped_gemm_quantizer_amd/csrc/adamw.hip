// An AdamW step over a list of tensors, with the gradients' clipping in it and the states in
// 32 bits or in 8.
//
//   g  = grad min(1, max_norm / (norm + 1e-6))         (where a sum of squares is given)
//   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2
//   p' = p (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v' / (1 - b2^t)) + eps)
//
// States in 8 bits: m and r = sqrt(v) (half the range of exponents to hold) as e4m3 codes, 128
// elements of a tensor to a power-of-two scale, the smallest that brings the block into range.
// A step moves v by 1 - b2 of its distance from g^2, far less than a code's step, so rounding to
// the nearest would leave it where it is: a value is rounded up with the probability of the part
// that is cut off, by 16 bits of a hash of (seed, step, tensor, element). r is never rounded to
// 0 unless it is 0: m / (r + eps) would then be as large as eps is small.
//
// An HBM stream: every tensor is read and written once (300 tensors of 50M, fp32 states, 241 to 250 us, 5.6 to
// 5.8 TB/s; 8 x 29M with 8-bit states 673, 5.6 TB/s). The list travels in the kernel's arguments, MAX_T tensors a
// launch, or lies in device memory for a launch over all of them (300 tensors of 50M: 6 launches 272 us, one
// 247; of 5M 54 / 27). Where the step's number or its rate lies on the device, every thread forms the factors in
// 64 bits: nothing beside fp32 states (300 tensors of 50M 252 us both ways, captured 274 / 272), 4% of a
// vector-bound step (8 x 29M with 8-bit states 706 / 676, captured 709 / 681; 2 x 50M bf16 205 / 195).

#include <math.h>
#include <vector>

#include "elem.h"
#include "internal.h"

namespace fp8g {
namespace {

using namespace elem;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int THREADS = 256;
constexpr int MAX_T = 52;
constexpr int BLOCK = 128;                             // elements of an 8-bit state that share a scale
constexpr int64_t CHUNK_MIN = 2048, CHUNK_MAX = 8192;  // elements of a chunk, multiples of 2048
constexpr int64_t LONG = int64_t(1) << 24;             // elements of a list that takes large chunks
constexpr int64_t CHUNKS = (1 << 24) - 1;              // of a launch: fewer than 2^32 threads
constexpr int64_t TABLE_CHUNKS = (int64_t(1) << 31) - 1;

struct Entry {
  void* p;
  const void* g;
  void* m;
  void* v;
  void* copy;
  uint8_t* ms;
  uint8_t* vs;
  int64_t numel;
  int first;                                           // the tensor's first chunk
  uint8_t types;                                       // of p + 3 of g
  uint8_t ctype;
};
static_assert(sizeof(Entry) == 72, "whole dwords");

struct Hyper {
  const double* sumsq;
  float* norm;                                         // written by this launch, or null
  const int64_t* step_at;
  const float* lr_at;
  double log1, log2, lr, decay;                        // log b1, log b2
  float b1, c1, b2, c2, eps, max_norm;                 // c1 = 1 - b1, c2 = 1 - b2
  int64_t step;
  uint32_t seed, key;
  float size, inv, keep;                               // Factors', where the host knows step and lr
};
// The chunk's tensor, c the same in all lanes.
template <typename Ends>
__device__ __forceinline__ int find_tensor(Ends end, int n, int c) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (c < end[mid]) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Tensors by value, from number `base` of the caller's list on; end: chunks of a tensor and those
// before it.
struct Some {
  Hyper h;
  int n, chunk, base;
  int end[MAX_T];
  Entry list[MAX_T];
  __device__ __forceinline__ int find(int c) const { return find_tensor(end, n, c); }
  __device__ __forceinline__ Entry at(int i) const { return list[i]; }
};
static_assert(sizeof(Some) <= 4096, "a kernel's arguments");

// All of them in device memory, a launch's chunks from number chunk0 on. The table is read through the
// scalar cache, which the tensors' stream does not pass (by vector loads, 64 ends at once, 300 tensors of
// 50M with 8-bit states took 190 us).
#define FP8G_CONSTANT __attribute__((address_space(4)))
struct All {
  Hyper h;
  int n, chunk, base, chunk0;
  const int* end;
  const Entry* list;
  __device__ __forceinline__ int find(int c) const {
    return find_tensor((const FP8G_CONSTANT int*)(uintptr_t)end, n, c);
  }
  __device__ __forceinline__ Entry at(int i) const {
    const FP8G_CONSTANT Entry* const e = (const FP8G_CONSTANT Entry*)(uintptr_t)(list + i);
    Entry o;
    o.p = e->p;
    o.g = e->g;
    o.m = e->m;
    o.v = e->v;
    o.copy = e->copy;
    o.ms = e->ms;
    o.vs = e->vs;
    o.numel = e->numel;
    o.first = e->first;
    o.types = e->types;
    o.ctype = e->ctype;
    return o;
  }
};
#undef FP8G_CONSTANT
template <typename A>
constexpr bool is_all = __is_same(A, All);
int64_t ends_bytes(int n) { return (n + 1) / 2 * 8; }

// What a step multiplies with, the same in every thread.
struct Factors {
  float clip, b1, c1, b2, c2, keep, size, inv, eps;    // keep = 1 - lr wd, size = lr / (1 - b1^t), inv = 1 / sqrt(1 - b2^t)
  uint32_t key;
};

// A 32-bit hash: xor-shifts and odd multipliers. (Shifts and multipliers as C. Wellons published them in 2018,
// found by a search for the least bias.)
__host__ __device__ __forceinline__ uint32_t mix(uint32_t h) {
  h = (h ^ (h >> 16)) * 0x7FEB352Du;
  h = (h ^ (h >> 15)) * 0x846CA68Bu;
  return h ^ (h >> 16);
}

// (1 - b^t without the cancellation at small t; b = 0 has log b = -inf)
template <typename O>
__host__ __device__ __forceinline__ void of_step(const Hyper& h, int64_t step, double lr, O& o) {
  o.size = (float)(lr / -expm1((double)step * h.log1));
  o.inv = (float)(1.0 / sqrt(-expm1((double)step * h.log2)));
  o.keep = (float)(1.0 - lr * h.decay);
  o.key = mix(h.seed + mix((uint32_t)step));
}

// (false: the sum of squares is infinite or NaN, and the step is left out)
__device__ __forceinline__ bool factors(const Hyper& h, Factors& f) {
  f.clip = 1.0f;
  if (h.sumsq) {
    const double norm = sqrt(*h.sumsq);
    if (h.norm && blockIdx.x == 0 && threadIdx.x == 0) *h.norm = (float)norm;
    if (!(norm < __builtin_inf())) return false;
    const double q = (double)h.max_norm / (norm + 1e-6);
    f.clip = q >= 1.0 ? 1.0f : (float)q;
  }
  if (h.step_at || h.lr_at) {
    of_step(h, h.step_at ? max(*h.step_at, (int64_t)1) : h.step, h.lr_at ? (double)*h.lr_at : h.lr, f);
  } else {
    f.size = h.size;
    f.inv = h.inv;
    f.keep = h.keep;
    f.key = h.key;
  }
  f.b1 = h.b1;
  f.c1 = h.c1;
  f.b2 = h.b2;
  f.c2 = h.c2;
  f.eps = h.eps;
  return true;
}

// One element's states. Products and sums are rounded one by one, so that their bits do not
// depend on which of them the compiler joins.
__device__ __forceinline__ void move(float g, float& m, float& v, const Factors& f) {
#pragma clang fp contract(off)
  g = g * f.clip;
  m = m * f.b1 + g * f.c1;
  v = v * f.b2 + g * g * f.c2;
}
// (the reciprocal within one ulp)
__device__ __forceinline__ float moved(float p, float m, float r, const Factors& f) {
#pragma clang fp contract(off)
  return p * f.keep - f.size * m * __builtin_amdgcn_rcpf(r * f.inv + f.eps);
}

// The square root, correctly rounded for every x from ROOT_MIN to below ROOT_END (compared on
// all of them): five instructions for the fourteen that the whole range takes.
constexpr float ROOT_MIN = 0x1p-96f, ROOT_END = 0x1p126f;
__device__ __forceinline__ float root(float x) {
#pragma clang fp contract(off)
  const float q = __builtin_amdgcn_rsqf(x), s = x * q;
  return __builtin_fmaf(__builtin_fmaf(-s, s, x), 0.5f * q, s);
}

// The square root within one ulp. The instruction takes a subnormal as 0, which with eps = 0 made an
// infinite step of a finite one: those are brought up by 2^64 first. (The stream hides these
// instructions: 300 tensors of 50M 245 us with and without them.)
__device__ __forceinline__ float root_of_state(float v) {
  const bool small = v < 0x1p-126f;
  return __builtin_amdgcn_sqrtf(small ? v * 0x1p64f : v) * (small ? 0x1p-32f : 1.0f);
}

// N values of type T as fp32: in 16-byte accesses (the address is aligned to what they move),
// or one by one, `left` of them.
template <typename T, int N>
struct Raw {
  static constexpr int W = N * (int)sizeof(T) < 16 ? N * (int)sizeof(T) / 4 : 4;       // dwords of an access
  static constexpr int K = N * (int)sizeof(T) / (4 * W);
  typedef uint32_t Word __attribute__((ext_vector_type(W)));
  Word w[K];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = __builtin_nontemporal_load(reinterpret_cast<const Word*>(p) + k);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int k = 0; k < K; ++k) __builtin_nontemporal_store(w[k], reinterpret_cast<Word*>(p) + k);
  }
  __device__ __forceinline__ void get(float (&x)[N]) const {
    const Pack<T, N> v = __builtin_bit_cast(Pack<T, N>, w);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(v.v[i]);
  }
  __device__ __forceinline__ void set(const float (&x)[N]) {
    Pack<T, N> v;
#pragma unroll
    for (int i = 0; i < N; ++i) v.v[i] = from_f32<T>(x[i]);
    __builtin_memcpy(&w, &v, sizeof(w));
  }
};
template <typename T, int N>
__device__ __forceinline__ void load_few(const T* p, int left, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = i < left ? to_f32(p[i]) : 0.0f;
}
template <typename T, int N>
__device__ __forceinline__ void store_few(T* p, int left, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < left) p[i] = from_f32<T>(x[i]);
}
template <int N>
__device__ __forceinline__ void store_copy(void* c, int64_t at, int type, bool vec, int left, const float (&x)[N]) {
  const auto put = [&](auto* p) __attribute__((always_inline)) {
    typedef __remove_reference_t(decltype(*p)) T;
    if (vec) {
      Raw<T, N> r;
      r.set(x);
      r.store(p + at);
    } else {
      store_few<T, N>(p + at, left, x);
    }
  };
  if (type == TYPE_BF16) put((bf16_t*)c);
  else put((f16_t*)c);
}

// A chunk with fp32 states: four elements a lane.
template <typename P, typename G>
__device__ __forceinline__ void chunk32(const Entry& t, int64_t at, int n, const Factors& f) {
  P* const p = (P*)t.p + at;
  const G* const g = (const G*)t.g + at;
  float* const m = (float*)t.m + at;
  float* const v = (float*)t.v + at;
  void* const c = t.copy;
  constexpr int N = 4;
  const bool vec = (((uintptr_t)p % (N * sizeof(P))) | ((uintptr_t)g % (N * sizeof(G))) |
                    (((uintptr_t)m | (uintptr_t)v) % 16) | ((uintptr_t)c % 8)) == 0;
#pragma unroll 2
  for (int e = threadIdx.x * N; e < n; e += THREADS * N) {
    float xp[N], xg[N], xm[N], xv[N];
    const int left = n - e;
    const bool whole = vec && left >= N;
    if (whole) {
      Raw<P, N> rp;
      Raw<G, N> rg;
      Raw<float, N> rm, rv;
      rp.load(p + e);
      rg.load(g + e);
      rm.load(m + e);
      rv.load(v + e);
      rp.get(xp);
      rg.get(xg);
      rm.get(xm);
      rv.get(xv);
    } else {
      load_few<P, N>(p + e, left, xp);
      load_few<G, N>(g + e, left, xg);
      load_few<float, N>(m + e, left, xm);
      load_few<float, N>(v + e, left, xv);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      move(xg[k], xm[k], xv[k], f);
      xp[k] = moved(xp[k], xm[k], root_of_state(xv[k]), f);
    }
    if (whole) {
      Raw<P, N> rp;
      Raw<float, N> rm, rv;
      rp.set(xp);
      rm.set(xm);
      rv.set(xv);
      rp.store(p + e);
      rm.store(m + e);
      rv.store(v + e);
    } else {
      store_few<P, N>(p + e, left, xp);
      store_few<float, N>(m + e, left, xm);
      store_few<float, N>(v + e, left, xv);
    }
    if (c) store_copy<N>(c, at + e, t.ctype, whole, left, xp);
  }
}

// The exponent of a block's scale: the smallest e with amax <= 448 2^e = 0.875 2^(e + 9), held
// to -126 and above; 0 for a block of zeros.
__device__ __forceinline__ int scale_exp(uint32_t amax) {
  const int e = (int)(amax >> 23) - 135 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax == 0u ? 0 : max(e, -126);
}
__device__ __forceinline__ float two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// |x| 2^-e (up to 448) as the lower 7 bits of an e4m3 code: 20 bits are cut off after 16 random
// ones are added above the lowest four (`cut`: already there). Below 2^-6, where a code's step
// stays 2^-9, 2^-6 is added first, which gives those values the same step, and taken off the code.
__device__ __forceinline__ uint32_t code7(float x, float scale, uint32_t cut) {
#pragma clang fp contract(off)
  const float z = __builtin_fabsf(x) * scale;
  const bool small = z < 0x1p-6f;
  const uint32_t u = __float_as_uint(z + (small ? 0x1p-6f : 0.0f));
  return (u + cut - ((small ? 968u : 960u) << 20)) >> 20;
}

// A chunk with states in 8 bits: eight elements a lane, 16 lanes a block.
template <typename P, typename G>
__device__ __forceinline__ void chunk8(const Entry& t, int index, int64_t at, int n, const Factors& f) {
  P* const p = (P*)t.p + at;
  const G* const g = (const G*)t.g + at;
  uint8_t* const m = (uint8_t*)t.m + at;
  uint8_t* const v = (uint8_t*)t.v + at;
  uint8_t* const ms = t.ms + at / BLOCK;
  uint8_t* const vs = t.vs + at / BLOCK;
  void* const c = t.copy;
  constexpr int N = 8;
  const bool vec = (((uintptr_t)p | (uintptr_t)g | (uintptr_t)c) % 16 | ((uintptr_t)m | (uintptr_t)v) % 8) == 0;
  const uint32_t key = mix(f.key + (uint32_t)index) + (uint32_t)(at / BLOCK);
  const int lane = threadIdx.x & 15;
  // (whole blocks: all 16 lanes of one take part in its maxima)
  for (int e = threadIdx.x * N; e - lane * N < n; e += THREADS * N) {
    float xp[N], xg[N];
    uint32_t cm[2] = {0, 0}, cv[2] = {0, 0};
    const int left = n - e, blk = e / BLOCK;
    const bool whole = vec && left >= N;
    const uint32_t sm = ms[blk], sv = vs[blk];
    if (whole) {
      Raw<P, N> rp;
      Raw<G, N> rg;
      Raw<uint32_t, 2> rm, rv;
      rp.load(p + e);
      rg.load(g + e);
      rm.load(reinterpret_cast<const uint32_t*>(m + e));
      rv.load(reinterpret_cast<const uint32_t*>(v + e));
      rp.get(xp);
      rg.get(xg);
      cm[0] = rm.w[0][0];
      cm[1] = rm.w[0][1];
      cv[0] = rv.w[0][0];
      cv[1] = rv.w[0][1];
    } else {
      load_few<P, N>(p + e, left, xp);
      load_few<G, N>(g + e, left, xg);
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < left) {
          cm[k / 4] |= (uint32_t)m[e + k] << (8 * (k % 4));
          cv[k / 4] |= (uint32_t)v[e + k] << (8 * (k % 4));
        }
    }
    const float fm = __uint_as_float(sm << 23), fv = __uint_as_float(sv << 23);
    float xm[N], xr[N];
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const auto dm = (k & 2) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)cm[k / 4], true)
                              : __builtin_amdgcn_cvt_pk_f32_fp8((int)cm[k / 4], false);
      const auto dv = (k & 2) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)cv[k / 4], true)
                              : __builtin_amdgcn_cvt_pk_f32_fp8((int)cv[k / 4], false);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        xm[k + h] = dm[h] * fm;
        xr[k + h] = dv[h] * fv;
      }
    }
    // (byte 255, which no step writes, is e8m0's NaN; a code of 0 is 0 under it as under every scale)
    if (max(sm, sv) == 255u) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const uint32_t bm = cm[k / 4] >> (8 * (k % 4)) & 0x7Fu, bv = cv[k / 4] >> (8 * (k % 4)) & 0x7Fu;
        if (sm == 255u) xm[k] = bm ? __builtin_nanf("") : 0.0f;
        if (sv == 255u) xr[k] = bv ? __builtin_nanf("") : 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      xr[k] = xr[k] * xr[k];
      move(xg[k], xm[k], xr[k], f);
    }
    float lo = xr[0], hi = xr[0];
#pragma unroll
    for (int k = 1; k < N; ++k) {
      lo = __builtin_fminf(lo, xr[k]);
      hi = __builtin_fmaxf(hi, xr[k]);
    }
    // (a NaN among them is dropped here, and root gives NaN for it as well)
    if (lo >= ROOT_MIN && hi < ROOT_END) {
#pragma unroll
      for (int k = 0; k < N; ++k) xr[k] = root(xr[k]);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) xr[k] = __builtin_sqrtf(xr[k]);
    }
    // (r is not negative, so that the patterns of both are in the values' order, infinities
    // and NaN above them)
    uint32_t am = 0, ar = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      xp[k] = moved(xp[k], xm[k], xr[k], f);
      am = max(am, __float_as_uint(xm[k]) << 1);
      ar = max(ar, __float_as_uint(xr[k]));
    }
    const auto umax = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    am = reduce_u32<16>(am, umax) >> 1;
    ar = reduce_u32<16>(ar, umax);
    const bool odd = am >= 0x7F800000u || ar >= 0x7F800000u;         // (the same in a block's lanes)
    if (odd) {
      am = ar = 0;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const uint32_t um = __float_as_uint(xm[k]) & 0x7FFFFFFFu, ur = __float_as_uint(xr[k]);
        am = max(am, um < 0x7F800000u ? um : 0u);
        ar = max(ar, ur < 0x7F800000u ? ur : 0u);
      }
      am = reduce_u32<16>(am, umax);
      ar = reduce_u32<16>(ar, umax);
    }
    const int em = scale_exp(am), er = scale_exp(ar);
    const uint32_t base = mix(key + (uint32_t)blk) + (uint32_t)(lane * N) * 0x9E3779B9u;
    const float im = two(-em), ir = two(-er);
    uint32_t om[2] = {0, 0}, ov[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t cut = mix(base + (uint32_t)k * 0x9E3779B9u);
      const uint32_t um = __float_as_uint(xm[k]), ur = __float_as_uint(xr[k]);
      uint32_t a = code7(xm[k], im, (cut & 0xFFFFu) << 4);
      uint32_t b = max(code7(xr[k], ir, (cut >> 12) & 0xFFFF0u), min(ur, 1u));
      if (odd) {
        a = (um & 0x7FFFFFFFu) < 0x7F800000u ? a : 0x7Fu;
        b = ur < 0x7F800000u ? b : 0x7Fu;
      }
      om[k / 4] |= (a | (um >> 24 & 0x80u)) << (8 * (k % 4));
      ov[k / 4] |= b << (8 * (k % 4));
    }
    if (whole) {
      Raw<P, N> rp;
      Raw<uint32_t, 2> rm, rv;
      rp.set(xp);
      rm.w[0][0] = om[0];
      rm.w[0][1] = om[1];
      rv.w[0][0] = ov[0];
      rv.w[0][1] = ov[1];
      rp.store(p + e);
      rm.store(reinterpret_cast<uint32_t*>(m + e));
      rv.store(reinterpret_cast<uint32_t*>(v + e));
    } else {
      store_few<P, N>(p + e, left, xp);
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < left) {
          m[e + k] = (uint8_t)(om[k / 4] >> (8 * (k % 4)));
          v[e + k] = (uint8_t)(ov[k / 4] >> (8 * (k % 4)));
        }
    }
    if (c) store_copy<N>(c, at + e, t.ctype, whole, left, xp);
    if (lane == 0) {
      ms[blk] = (uint8_t)(em + 127);
      vs[blk] = (uint8_t)(er + 127);
    }
  }
}

// A workgroup a chunk (n == 0: one writes the norm).
template <int BITS, typename Args>
__global__ void __launch_bounds__(THREADS)
adamw_kernel(Args a) {
  Factors f;
  if (!factors(a.h, f)) return;
  if (a.n == 0) return;
  int c = (int)blockIdx.x;
  if constexpr (is_all<Args>) c += a.chunk0;
  const int i = a.find(c);
  const Entry t = a.at(i);
  const int64_t at = (int64_t)(c - t.first) * a.chunk;
  const int64_t left = t.numel - at;
  const int n = (int)(left < a.chunk ? left : a.chunk);
  const auto run = [&](auto p, auto g) __attribute__((always_inline)) {
    if constexpr (BITS == 8) chunk8<decltype(p), decltype(g)>(t, a.base + i, at, n, f);
    else chunk32<decltype(p), decltype(g)>(t, at, n, f);
  };
  switch (t.types) {
    case 0: run(0.0f, 0.0f); break;
    case 1: run(bf16_t(), 0.0f); break;
    case 2: run(f16_t(), 0.0f); break;
    case 3: run(0.0f, bf16_t()); break;
    case 4: run(bf16_t(), bf16_t()); break;
    case 5: run(f16_t(), bf16_t()); break;
    case 6: run(0.0f, f16_t()); break;
    case 7: run(bf16_t(), f16_t()); break;
    default: run(f16_t(), f16_t()); break;
  }
}

// A list's chunk. Small ones where HBM is the bound: they reach all CUs and end evenly (2048 /
// 8192 elements: 300 tensors of 50M, fp32 parameters, fp32 states 246 / 277 us, 8-bit states 142 /
// 166; 8 x 29M 8-bit 672 / 741; 3M elements 13.7 / 16.4; 300 bf16 tensors of 5M 18.7 / 21.3). Large lists of
// 16-bit parameters with 8-bit states are bound by the vector unit, which what a workgroup does once (the
// clipping factor in fp64, the search) keeps busy too (2 x 50M bf16 208 / 195, 300 of 50M 108 / 102, of 17M 44 / 43).
int chunk_for(const AdamwCall& c) {
  if (!c.ms) return CHUNK_MIN;
  int64_t total = 0, narrow = 0;
  for (int i = 0; i < c.n; ++i) {
    total += c.numels[i];
    if (c.param_types[i] != TYPE_F32) narrow += c.numels[i];
  }
  return (int)(total >= LONG && narrow > total / 2 ? CHUNK_MAX : CHUNK_MIN);
}

int64_t chunks_of(int64_t numel, int chunk) { return (numel + chunk - 1) / chunk; }

// Tensor i's entry, its chunks from `first` on.
Entry entry(const AdamwCall& c, int i, int64_t first) {
  Entry e = {};
  e.p = c.params[i];
  e.g = c.grads[i];
  e.m = c.m[i];
  e.v = c.v[i];
  e.copy = c.copies ? c.copies[i] : nullptr;
  e.ms = c.ms ? c.ms[i] : nullptr;
  e.vs = c.ms ? c.vs[i] : nullptr;
  e.numel = c.numels[i];
  e.first = (int)first;
  e.types = (uint8_t)(c.param_types[i] + 3 * c.grad_types[i]);
  e.ctype = (uint8_t)(c.copies ? c.copy_types[i] : 0);
  return e;
}

Hyper hyper(const AdamwCall& c) {
  Hyper h = {};
  h.sumsq = c.sumsq;
  h.norm = c.norm;
  h.step_at = c.step_at;
  h.lr_at = c.lr_at;
  h.log1 = log(c.beta1);
  h.log2 = log(c.beta2);
  h.lr = c.lr;
  h.decay = c.weight_decay;
  h.b1 = (float)c.beta1;
  h.c1 = (float)(1.0 - c.beta1);
  h.b2 = (float)c.beta2;
  h.c2 = (float)(1.0 - c.beta2);
  // (the reciprocal of a subnormal is infinite, and an element without gradient and states then NaN)
  h.eps = c.eps > 0.0 && c.eps < 0x1p-126 ? 0x1p-126f : (float)c.eps;
  h.max_norm = c.max_norm;
  h.step = c.step;
  h.seed = c.seed;
  if (!c.step_at && !c.lr_at) of_step(h, c.step, c.lr, h);
  return h;
}

hipError_t launch_all(const AdamwCall& c, hipStream_t stream) {
  All a;
  a.h = hyper(c);
  a.n = c.n;
  a.chunk = chunk_for(c);
  a.base = 0;
  a.end = (const int*)c.table;
  a.list = (const Entry*)((const char*)c.table + ends_bytes(c.n));
  int64_t chunks = 0;
  for (int i = 0; i < c.n; ++i) chunks += chunks_of(c.numels[i], a.chunk);
  const auto kernel = c.ms ? adamw_kernel<8, All> : adamw_kernel<32, All>;
  for (int64_t at = 0; at < chunks; at += CHUNKS) {
    a.chunk0 = (int)at;
    kernel<<<dim3((unsigned)(chunks - at < CHUNKS ? chunks - at : CHUNKS)), dim3(THREADS), 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.h.norm = nullptr;
  }
  return hipSuccess;
}

hipError_t launch_some(const AdamwCall& c, hipStream_t stream) {
  Some a;
  a.h = hyper(c);
  a.chunk = chunk_for(c);
  const auto kernel = c.ms ? adamw_kernel<8, Some> : adamw_kernel<32, Some>;
  int i = 0;
  bool first = true;
  for (;;) {
    a.n = 0;
    a.base = i;
    int64_t chunks = 0;
    for (; i < c.n && a.n < MAX_T; ++i) {
      const int64_t k = chunks_of(c.numels[i], a.chunk);
      if (chunks + k > CHUNKS && a.n > 0) break;       // (each tensor fits by itself: checked before)
      a.list[a.n] = entry(c, i, chunks);
      chunks += k;
      a.end[a.n] = (int)chunks;
      ++a.n;
    }
    if (chunks == 0) a.n = 0;
    // (nothing to do, but a norm to write)
    if (chunks > 0 || (first && c.norm)) {
      kernel<<<dim3((unsigned)(chunks ? chunks : 1)), dim3(THREADS), 0, stream>>>(a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      a.h.norm = nullptr;
      first = false;
    }
    if (i >= c.n) break;
  }
  return hipSuccess;
}

}  // namespace

size_t adamw_table_bytes(int n) { return (size_t)ends_bytes(n) + (size_t)n * sizeof(Entry); }

bool adamw_table_fill(const AdamwCall& c, void* table) {
  int* const end = (int*)table;
  Entry* const list = (Entry*)((char*)table + ends_bytes(c.n));
  const int chunk = chunk_for(c);
  int64_t chunks = 0;
  for (int i = 0; i < c.n; ++i) {
    list[i] = entry(c, i, chunks);
    chunks += chunks_of(c.numels[i], chunk);
    if (chunks > TABLE_CHUNKS) return false;
    end[i] = (int)chunks;
  }
  if (c.n % 2) end[c.n] = 0;
  return true;
}

hipError_t launch_adamw(const AdamwCall& c, hipStream_t stream) {
  // (a graph holds what its launches were given: a list by value outlives the caller's table)
  if (c.table && c.n > MAX_T) {
    hipStreamCaptureStatus status;
    const hipError_t e = hipStreamIsCapturing(stream, &status);
    if (e != hipSuccess) return e;
    int64_t total = 0;
    for (int i = 0; i < c.n; ++i) total += c.numels[i];
    if (status == hipStreamCaptureStatusNone && total > 0) return launch_all(c, stream);
  }
  return launch_some(c, stream);
}

void adamw_kernels(std::vector<const void*>& out) {
  out.push_back((const void*)adamw_kernel<8, Some>);
  out.push_back((const void*)adamw_kernel<32, Some>);
  out.push_back((const void*)adamw_kernel<8, All>);
  out.push_back((const void*)adamw_kernel<32, All>);
}

}  // namespace fp8g
