// What the two routings share (softmax with the choice by logits; scores with a bias and
// groups): how a row lies over lanes, the choice of the largest values, offsets, loss, the ranks
// inside a block. Each of their files includes this once.
#pragma once

#include <type_traits>

#include "elem.h"
#include "internal.h"

namespace fp8g {
namespace {

using namespace elem;

constexpr int ROWS = 64;          // tokens of a block
constexpr int THREADS = 256;       // of a workgroup, where nothing else is said
constexpr int MAX_E = 1024;
constexpr int MAX_K = 16;

// Where a lane's VPT elements of a row lie: groups of W consecutive ones
// (one access), LPR lanes side by side.
template <typename T, int LPR, int VPT>
struct Lay {
  static constexpr int WMAX = 16 / (int)sizeof(T);
  static constexpr int W = VPT % WMAX == 0 ? WMAX : (VPT % 4 == 0 ? 4 : VPT);
  static_assert(VPT % W == 0 && W <= WMAX, "whole groups");
  __device__ static __forceinline__ int at(int v, int l) {
    return (v / W) * (W * LPR) + l * W + v % W;
  }
};

// A row's logits as fp32; past E (and for a row that takes no part) -inf.
template <typename T, int LPR, int VPT>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int E, int l, bool on, bool vec,
                                         float (&x)[VPT]) {
  using L = Lay<T, LPR, VPT>;
#pragma unroll
  for (int g = 0; g < VPT / L::W; ++g) {
    const int e0 = L::at(g * L::W, l);
    if (vec && on && e0 + L::W <= E) {
      const Pack<T, L::W> p = *reinterpret_cast<const Pack<T, L::W>*>(row + e0);
#pragma unroll
      for (int w = 0; w < L::W; ++w) x[g * L::W + w] = to_f32(p.v[w]);
    } else {
#pragma unroll
      for (int w = 0; w < L::W; ++w)
        x[g * L::W + w] = on && e0 + w < E ? to_f32(row[e0 + w]) : -__builtin_inff();
    }
  }
}

// Unsigned keys in the order of the values (-0 as +0); 0 for what is never
// chosen: -inf and NaN.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return x > -__builtin_inff() ? k : 0u;
}

// The largest remaining logit of each row, one after the other.
//
// A key holds the order of a value in its upper bits and, inverted, the
// expert's number below, so that one maximum finds the value and the lowest
// expert that has it, and all keys differ. The next one is the largest key
// below the last: with d = key - last in wrapping arithmetic, every key below
// it has a larger d than every key from it on, so it is last + max d, at one
// subtraction and half a three-way maximum per expert; no key is removed.
//
// 16-bit values fit a key whole. Of a 32-bit value BITS low bits give way to
// the expert's number: exact where they are zero in the whole row (values that
// were 16-bit ones, for instance); otherwise neighbours whose kept bits agree
// are not known to be in order, and `choose` puts them in order.
template <typename T, int LPR, int VPT>
struct Picker {
  using L = Lay<T, LPR, VPT>;
  static constexpr bool WHOLE = sizeof(T) == 2;
  static constexpr int BITS = WHOLE ? 16 : (LPR * VPT <= 256 ? 8 : 10);
  static constexpr uint32_t LOW = (1u << BITS) - 1u;
  uint32_t key[VPT];
  uint32_t last;
  uint32_t dropped;      // nonzero: bits of the row's values are not in its keys

  // (a 16-bit value's fp32 key: bf16 has its order in the upper half; fp16
  // is widened, so it is brought back to its own 16 bits)
  __device__ static __forceinline__ uint32_t upper(float x) {
    if constexpr (std::is_same<T, f16_t>::value) {
      const uint16_t u = __builtin_bit_cast(uint16_t, (f16_t)(x + 0.0f));
      const uint32_t k = (u & 0x8000u) ? (uint16_t)~u : (uint16_t)(u | 0x8000u);
      return x > -__builtin_inff() ? k << 16 : 0u;
    } else {
      return order_key(x) & ~LOW;
    }
  }

  __device__ __forceinline__ void start(const float (&x)[VPT], int l) {
    last = 0u;
    dropped = 0u;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const uint32_t h = upper(x[v]);
      key[v] = h ? h | (LOW - (uint32_t)L::at(v, l)) : 0u;
      if constexpr (!WHOLE) dropped |= __float_as_uint(x[v]);
    }
    if constexpr (!WHOLE)
      dropped = reduce_u32<LPR>(dropped & LOW, [](uint32_t a, uint32_t b) { return a | b; });
  }
  // (the first call: everything lies below 2^32)
  __device__ __forceinline__ uint32_t next() {
    const auto umax = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    uint32_t d = key[0] - last;
#pragma unroll
    for (int v = 1; v < VPT; ++v) d = umax(d, key[v] - last);
    d = reduce_u32<LPR>(d, umax);
    const uint32_t k = last + d;
    // (none left below: d is one of the keys from `last` on; a key of 0 is
    // what is never chosen. `last` stays where it is then.)
    const bool none = k == 0u || (last != 0u && k >= last);
    last = none ? last : k;
    return none ? 0u : k;
  }
  __device__ static __forceinline__ int expert(uint32_t k) { return k ? (int)(LOW - (k & LOW)) : -1; }
};

// The k largest of whole 32-bit values: the value, then the lowest expert
// that has it, which is removed. Lane j gets the j-th.
template <int LPR, int VPT>
__device__ __forceinline__ int exact_choice(const float (&x)[VPT], int l, int k) {
  using L = Lay<float, LPR, VPT>;
  uint32_t key[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) key[v] = order_key(x[v]);
  int id = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < VPT; ++v) best = best > key[v] ? best : key[v];
    best = reduce_u32<LPR>(best, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    uint32_t low = 0xFFFFFFFFu;
#pragma unroll
    for (int v = VPT - 1; v >= 0; --v) low = key[v] == best ? (uint32_t)L::at(v, l) : low;
    low = reduce_u32<LPR>(low, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
#pragma unroll
    for (int v = 0; v < VPT; ++v) key[v] = (uint32_t)L::at(v, l) == low ? 0u : key[v];
    if (l == j && best) id = (int)low;
  }
  return id;
}

// Lane j gets the row's j-th choice (-1: none) and its logit, of which `row` is
// the first.
template <typename T, int LPR, int VPT>
__device__ __forceinline__ int choose(const float (&x)[VPT], const T* __restrict__ row, int l, int k,
                                      float& value) {
  using P = Picker<T, LPR, VPT>;
  P pick;
  pick.start(x, l);
  uint32_t mine = 0u, before = 0u;
  bool close = false;
  for (int j = 0; j < k; ++j) {
    const uint32_t key = pick.next();
    if constexpr (!P::WHOLE) close = close || (key && ((key ^ before) >> P::BITS) == 0u);
    before = key;
    if (l == j) mine = key;
  }
  int id = P::expert(mine);
  // (the row was just read: its value again is a cache hit)
  value = id >= 0 ? to_f32(row[id]) : 0.0f;
  if constexpr (!P::WHOLE) {
    if (__ballot(pick.dropped != 0u)) {                // (uniform over the wave, as all of these)
      const uint32_t key = pick.next();
      const bool edge = key && ((key ^ before) >> P::BITS) == 0u;
      if (__ballot(edge && pick.dropped != 0u)) {
        // the k-th and the next one: which of them is larger, or a third
        id = exact_choice<LPR, VPT>(x, l, k);
        value = id >= 0 ? to_f32(row[id]) : 0.0f;
      } else if (__ballot(close && pick.dropped != 0u)) {
        // neighbours among the chosen: exchanged until whole values are in
        // order (most often two of them, once)
        uint32_t full = id >= 0 ? order_key(value) : 0u;
        bool moved;
        do {
          moved = false;
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const int with = ((l + odd) ^ 1) - odd;
            const bool first = with > l, pair = l < MAX_K && with >= 0 && with < MAX_K;
            const uint32_t f = (uint32_t)__shfl((int)full, with & (LPR - 1), LPR);
            const int i = __shfl(id, with & (LPR - 1), LPR);
            const float v = __shfl(value, with & (LPR - 1), LPR);
            // (0: no choice; two of those stay where they are)
            const bool ahead = f > full || (f == full && i < id);    // the other one is
            if (pair && (f | full) != 0u && ahead == first) {
              full = f;
              id = i;
              value = v;
              moved = true;
            }
          }
        } while (__ballot(moved));
      }
    }
  }
  return id;
}

// exp(x - max) of a row and their sum's reciprocal. A row of -inf alone has
// p = 0; NaN or +inf in a row make its p NaN.
template <int LPR, int VPT>
__device__ __forceinline__ float row_softmax(const float (&x)[VPT], float& top, float (&ex)[VPT]) {
  float m = x[0];
#pragma unroll
  for (int v = 1; v < VPT; ++v) m = __builtin_fmaxf(m, x[v]);
  m = max_lanes<LPR>(m);
  top = m > -__builtin_inff() ? m : 0.0f;        // (m is NaN for a row of NaN alone)
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    ex[v] = exp_neg(x[v] - top);
    s += ex[v];
  }
  s = sum_lanes<LPR>(s);
  return s == 0.0f ? 0.0f : 1.0f / s;
}

// Expert offsets of the contiguous layout: exclusive prefix sums of the
// counts rounded up to `align`, by the NT threads of the workgroup.
template <int NT>
__device__ __forceinline__ void offsets_of(const int* __restrict__ counts, int E, int align,
                                           int* __restrict__ off, int* __restrict__ wave_sum) {
  constexpr int PER = MAX_E / NT;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int c[PER], s = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = t * PER + i;
    c[i] = e < E ? (counts[e] + align - 1) / align * align : 0;
    s += c[i];
  }
  int inc = s;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 63) wave_sum[wave] = inc;
  __syncthreads();
  int at = inc - s;
  for (int w = 0; w < wave; ++w) at += wave_sum[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = t * PER + i;
    if (e < E) off[e] = at;
    at += c[i];
    if (e == E - 1) off[E] = at;
  }
  __syncthreads();
}

// loss = coef sum_e (E c_e / (k n)) (P_e / n), by one wave.
__device__ __forceinline__ void write_loss(const int* counts, const float* prob_sum, int routed,
                                           int E, int k, float coef, float* loss) {
  const int lane = threadIdx.x & 63;
  double s = 0.0;
  for (int e = lane; e < E; e += 64) s += (double)counts[e] * (double)prob_sum[e];
  s = sum_wave(s);
  const double n = routed > 0 ? (double)routed : 1.0;
  if (lane == 0) *loss = (float)((double)coef * E / ((double)k * n * n) * s);
}

struct RouteArgs {
  const void* logits;
  const uint8_t* mask;
  int64_t T, ld, max_m;
  int E, k, renorm, align, vec;
  int block0, only;                 // this launch's first block; whether it is the only one of all
  float coef;
  int32_t *ids, *counts, *routed, *offsets, *slots;
  float *weights, *prob_sum, *loss;
  // one row of counts (the routed tokens last) and of sums of p per block
  int* part_count;
  float* part_prob;
};

__device__ __forceinline__ int slot_of(const RouteArgs& a, int e, int first, int rank) {
  if (a.max_m == 0) return first + rank;
  return rank < a.max_m ? (int)(e * a.max_m) + rank : -1;
}

// What is left of a block's work when its tokens have chosen: `acc` is what a lane's rows added to
// its experts' sums of probabilities, `took` holds the block's tokens that chose each expert as
// bits, `chosen` the experts of each row. Counts and sums go out (and, where the block is the
// only one, offsets and loss), and the ranks inside the block.
template <typename T, int LPR, int VPT, int NT>
__device__ __forceinline__ void finish_block(const RouteArgs& a, int64_t block, float (&acc)[VPT],
                                             uint32_t (&took)[2][MAX_E], short (&chosen)[ROWS][MAX_K],
                                             float (&psum)[NT / 64][LPR * VPT], int (&count)[MAX_E],
                                             int (&off)[MAX_E + 1], int (&wave_sum)[NT / 64], int& n_routed) {
  using L = Lay<T, LPR, VPT>;
  constexpr int GROUPS = 64 / LPR, WAVES = NT / 64;
  const int E = a.E, k = a.k;
  const int l = threadIdx.x & (LPR - 1), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t0 = block * ROWS;
  // sums of p: the rows side by side in a wave, then the waves
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if constexpr (GROUPS > 1) {
      const uint32_t u = __float_as_uint(acc[v]);
      const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
      const uint32_t w = __float_as_uint(__uint_as_float(p[0]) + __uint_as_float(p[1]));
      const auto q = __builtin_amdgcn_permlane32_swap(w, w, false, false);
      acc[v] = __uint_as_float(q[0]) + __uint_as_float(q[1]);
    }
    if (lane < LPR) psum[wave][L::at(v, l)] = acc[v];
  }
  __syncthreads();
  const bool only = a.only != 0;
  for (int e = threadIdx.x; e < E; e += NT) {
    const int c = __popc(took[0][e]) + __popc(took[1][e]);
    float p = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; w += 4)
      p += (psum[w][e] + psum[w + 1][e]) + (psum[w + 2][e] + psum[w + 3][e]);
    if (only) {
      a.counts[e] = c;
      a.prob_sum[e] = p;
      psum[0][e] = p;
      count[e] = c;
    } else {
      a.part_count[block * (E + 1) + e] = c;
      a.part_prob[block * E + e] = p;
    }
  }
  if (threadIdx.x == 0) {
    if (only) a.routed[0] = n_routed;
    else a.part_count[block * (E + 1) + E] = n_routed;
  }
  if (only) {
    __syncthreads();
    if (a.max_m == 0) {
      offsets_of<NT>(count, E, a.align, off, wave_sum);
      for (int e = threadIdx.x; e <= E; e += NT) a.offsets[e] = off[e];
    } else {
      for (int e = threadIdx.x; e <= E; e += NT) a.offsets[e] = (int)(e * a.max_m);
    }
    if (wave == WAVES - 1) write_loss(count, psum[0], n_routed, E, k, a.coef, a.loss);
  }
  // ranks inside the block (its only block: the slots themselves)
  const int64_t left = a.T - t0;
  const int rows = left < ROWS ? (int)left : ROWS;
  for (int i = threadIdx.x; i < rows * k; i += NT) {
    const int r = i / k, e = chosen[r][i - r * k];
    int s = -1;
    if (e >= 0) {
      const uint32_t below = (1u << (r & 31)) - 1u;
      s = r < 32 ? __popc(took[0][e] & below)
                 : __popc(took[0][e]) + __popc(took[1][e] & below);
      if (only) s = slot_of(a, e, off[e], s);
    }
    a.slots[t0 * k + i] = s;
  }
}

// Orders a wave's LDS accesses for the compiler (the LDS itself takes them in
// order).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

bool vec_ok(const void* p, int64_t ld, int type) {
  const int64_t size = type == TYPE_F32 ? 4 : 2;
  return (uintptr_t)p % 16 == 0 && ld * size % 16 == 0;
}

// The kernels' arguments of a call.
RouteArgs route_args(const RouteCall& c) {
  RouteArgs a;
  a.logits = c.logits;
  a.mask = c.mask;
  a.T = c.T;
  a.ld = c.ld;
  a.max_m = c.max_m;
  a.E = c.E;
  a.k = c.k;
  a.renorm = c.renorm;
  a.align = c.align;
  a.vec = vec_ok(c.logits, c.ld, c.type);
  a.coef = c.coef;
  a.ids = c.ids;
  a.counts = c.counts;
  a.routed = c.routed;
  a.offsets = c.offsets;
  a.slots = c.slots;
  a.weights = c.weights;
  a.prob_sum = c.prob_sum;
  a.loss = c.loss;
  const int64_t nblk = (c.T + ROWS - 1) / ROWS;
  a.part_count = (int*)c.workspace;
  a.part_prob = nblk > 1 ? (float*)((char*)c.workspace +
                                    ((size_t)nblk * (c.E + 1) * sizeof(int) + 15) / 16 * 16)
                         : nullptr;
  a.block0 = 0;
  a.only = nblk == 1;
  return a;
}

// Workgroups of a launch: its threads are counted in 32 bits.
int64_t rows_blocks_max(int threads) { return 0xFFFFFFFFll / threads; }

}  // namespace
}  // namespace fp8g
