// Routing by scores: sigmoid or softmax of the logits, the experts chosen by score plus a bias
// that keeps them evenly loaded, inside the groups of experts whose best values' sum is largest;
// weights from the scores without the bias. The gradient of weights and balance loss.
//
//   s = sigmoid(x) or softmax(x);  v = s + b;  a group's value is the sum of its `best` (1 or 2)
//   largest v; the `open` groups of largest value are open; ids: the k largest v in them, ties to
//   the lower expert;  w = scale s[id] (over the sum of the chosen s);
//   loss = coef sum_e (E c_e / (k n)) (P_e / n), P_e the sum over tokens of s_e / sum s.
// With every group open and no bias the choice goes by the logits themselves (both scores rise
// with them), as in route.hip, whose scan and slots follow here too.
//
// Which of two values is larger is decided exactly: as in 64 bits. The fp32 values choose, as
// whole numbers of 24 (22) bits of the row's range with the expert's number below; where two
// neighbours among the chosen and the next, or the last open and the first closed group, are
// nearer than their errors and not alike (the same logit and bias), the row is put on a list and
// done again in 64 bits by a wave of its own: about 0.1% of the rows of random fp32 logits. It is most rows
// where a large bias (or, without biases and groups, a large logit) makes the range so wide that its unit
// is the scores' differences, and all rows where groups are alike. T 32768, E 256, fp32: 42 us, with eight experts
// closed by a bias of -inf or -10 41, of -1e4 114, of -1e9 115; without groups 34, 34, 87 and 100; closed by a
// logit, without biases, -inf 33, -1e4 53, -1e9 85; all logits and biases alike 118.
//
// T 32768, E 256, 8 groups, fp32: 31 us for the rows (the data 7.4 at the rate of a large copy), bound by the
// vector unit (1400 instructions for four rows, 18 us) and at the end by the rows done again, which take 6 us
// whether few or many: every block is on a CU from the start, and some have such a row. Then 12 for scan and
// slots.

#include <vector>

#include "route_common.h"

namespace fp8g {
namespace {

constexpr uint32_t MAX_GROUPS = 32;

struct ScoredArgs {
  RouteArgs r;
  const float* bias;
  int score, groups, open, best, size;                 // size: experts of a group
  uint32_t per_size;                                   // e / size = e per_size >> 20
  int part_bits, part_bits64;                          // 1 << these lanes a group, of a row's and of a wave's
  float scale;
};

// Sums of scores below this are formed again from exponentials shifted by the largest logit: both
// scores are exp(x) times a factor of the row there (sigmoid to 2^-32), and shares of a sum do not
// depend on it. A share of 2^-94 and above is as exact as the others, however far below fp32's range
// the scores are.
constexpr float LITTLE = 0x1p-32f;

// A row's scores, and what of them its share of the loss is: 1 / sum s (0 for a row without any,
// NaN where a logit is NaN, or with softmax infinite).
struct RowSum {
  float share, top, norm;                              // softmax: s = exp(x - top) norm
};
// sigmoid from exp(-|x|), exact to 4 ulp at both ends; and what it lacks of 1.
__device__ __forceinline__ float sigmoid(float x) {
  const float t = exp_neg(-__builtin_fabsf(x));
  return (x >= 0.0f ? 1.0f : t) * __builtin_amdgcn_rcpf(1.0f + t);
}
__device__ __forceinline__ float sigmoid(float x, float& rest) {
  const float t = exp_neg(-__builtin_fabsf(x)), q = __builtin_amdgcn_rcpf(1.0f + t), p = t * q;
  rest = x >= 0.0f ? p : q;
  return x >= 0.0f ? q : p;
}
template <int LPR, int VPT>
__device__ __forceinline__ RowSum row_scores(const float (&x)[VPT], int score, float (&s)[VPT]) {
  RowSum r;
  if (score == SCORE_SOFTMAX) {
    r.norm = row_softmax<LPR, VPT>(x, r.top, s);
#pragma unroll
    for (int v = 0; v < VPT; ++v) s[v] *= r.norm;
    r.share = r.norm > 0.0f ? 1.0f : r.norm;           // (0 and NaN stay)
  } else {
    float z = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      s[v] = sigmoid(x[v]);
      z += s[v];
    }
    z = sum_lanes<LPR>(z);
    r.share = z == 0.0f ? 0.0f : 1.0f / z;
    r.top = r.norm = 0.0f;
  }
  return r;
}
__device__ __forceinline__ float score_of(float x, int score, const RowSum& r) {
  return score == SCORE_SOFTMAX ? exp_neg(x - r.top) * r.norm : sigmoid(x);
}
// A row whose sigmoids are all little: s and share by shifted exponentials.
template <int LPR, int VPT>
__device__ __forceinline__ void little_scores(const float (&x)[VPT], bool little, float (&s)[VPT], float& share) {
  if (__ballot(little) == 0) return;                   // (uniform over the wave)
  float e[VPT], top;
  const float norm = row_softmax<LPR, VPT>(x, top, e);
#pragma unroll
  for (int v = 0; v < VPT; ++v) s[v] = little ? e[v] : s[v];
  share = little ? norm : share;
}
// The chosen scores' shares of their sum, each lane its own (`on`: it has one).
template <int LPR>
__device__ __forceinline__ float chosen_share(float s, float x, bool on) {
  float z = sum_lanes<LPR>(on ? s : 0.0f);
  const bool little = z < LITTLE;
  if (__ballot(little && on)) {
    const float top = max_lanes<LPR>(on ? x : -__builtin_inff());
    const float e = on ? exp_neg(x - top) : 0.0f;
    const float ze = sum_lanes<LPR>(e);
    s = little ? e : s;
    z = little ? ze : z;
  }
  return on ? s / z : 0.0f;
}

// Largest of a wave's values in 64 bits, in all lanes (by lane exchanges that do not go through LDS:
// a row that is done again is one chain of these, and its workgroup waits for it).
template <class F>
__device__ __forceinline__ double both_words(double x, F f) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  return __builtin_bit_cast(double, (uint64_t)f((uint32_t)u) | (uint64_t)f((uint32_t)(u >> 32)) << 32);
}
__device__ __forceinline__ double max_wave(double x) {
  x = fmax(x, both_words(x, [](uint32_t w) { return ring16<8>(w); }));
  x = fmax(x, both_words(x, [](uint32_t w) { return ring16<4>(w); }));
  x = fmax(x, both_words(x, [](uint32_t w) { return ring16<2>(w); }));
  x = fmax(x, both_words(x, [](uint32_t w) { return ring16<1>(w); }));
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const auto words = [](uint32_t lo, uint32_t hi) { return __builtin_bit_cast(double, (uint64_t)lo | (uint64_t)hi << 32); };
  const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
  x = fmax(words(lo[0], hi[0]), words(lo[1], hi[1]));
  const uint64_t w = __builtin_bit_cast(uint64_t, x);
  const auto lo2 = __builtin_amdgcn_permlane32_swap((uint32_t)w, (uint32_t)w, false, false);
  const auto hi2 = __builtin_amdgcn_permlane32_swap((uint32_t)(w >> 32), (uint32_t)(w >> 32), false, false);
  return fmax(words(lo2[0], hi2[0]), words(lo2[1], hi2[1]));
}

// One row by a wave in 64 bits: lane l holds experts l, l + 64, ... Lane j gets the j-th choice
// (-1: none), its logit and its score. few: the k + 1 experts among which the choice surely is, or all are looked
// at (null). high, low: LDS of the wave's own, a word each for every expert; 1 << part_bits
// lanes a group.
template <typename T, int PER>
__device__ __forceinline__ int choose64(const T* __restrict__ row, const ScoredArgs& a, int l, const short* few,
                                        uint32_t* high, uint32_t* low, int part_bits, float& xj, double& score) {
  const int E = a.r.E, k = a.r.k;
  const double none = -__builtin_inf();
  double v[PER], top = none, z = 1.0;
  if (!few || a.score == SCORE_SOFTMAX) {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = l + 64 * q;
      v[q] = e < E ? (double)to_f32(row[e]) : none;
      top = fmax(top, v[q]);
    }
  }
  // (loaded beside the row's: what follows is one chain)
  const int fe = few && l <= k ? few[l] : -1;
  const float fx = fe >= 0 ? to_f32(row[fe]) : 0.0f, fb = fe >= 0 && a.bias ? a.bias[fe] : 0.0f;
  if (a.score == SCORE_SOFTMAX) {
    top = max_wave(top);
    top = top > none ? top : 0.0;
    z = 0.0;
#pragma unroll
    for (int q = 0; q < PER; ++q) z += l + 64 * q < E ? exp(v[q] - top) : 0.0;
    z = sum_wave(z);
  }
  const auto score64 = [&](double x) __attribute__((always_inline)) {
    return a.score == SCORE_SOFTMAX ? exp(x - top) / z : 1.0 / (1.0 + exp(-x));
  };
  const bool by_value = a.bias || a.open < a.groups;
  if (few) {
    const double s64 = score64((double)fx);
    const double y = fe < 0 ? none : (a.bias ? s64 + (double)fb : (double)fx);
    const uint64_t words = __builtin_bit_cast(uint64_t, y);
    int rank = 0;
    for (int i = 0; i <= k; ++i) {
      const double o = __builtin_bit_cast(
          double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)words, i) |
                      (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(words >> 32), i) << 32);
      const int oe = __builtin_amdgcn_readlane(fe, i);
      rank += o > y || (o == y && oe < fe) ? 1 : 0;
    }
    // (each candidate's place is its rank)
    if (l < k) low[l] = 0xFFFFFFFFu;
    wave_sync();
    if (fe >= 0 && rank < k) low[rank] = (uint32_t)l;
    wave_sync();
    const int from = l < k ? (int)low[l] : -1;
    wave_sync();
    // (by all lanes: a lane that takes nothing may give)
    const int id = __shfl(fe, from & 63);
    const float xs = __shfl(fx, from & 63);
    const double ss = __shfl(s64, from & 63);
    xj = from >= 0 ? xs : 0.0f;
    score = from >= 0 ? ss : 0.0;
    return from >= 0 ? id : -1;
  }
  if (by_value) {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = l + 64 * q;
      const double y = score64(v[q]) + (a.bias && e < E ? (double)a.bias[e] : 0.0);
      v[q] = v[q] > none && y > none ? y : none;       // (NaN: neither)
    }
  } else {
#pragma unroll
    for (int q = 0; q < PER; ++q) v[q] = v[q] > none ? v[q] : none;
  }
  if (a.open < a.groups) {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = l + 64 * q;
      const uint64_t u = __builtin_bit_cast(uint64_t, v[q]);
      if (e < E) {
        high[e] = (uint32_t)(u >> 32);
        low[e] = (uint32_t)u;
      }
    }
    wave_sync();
    const int g = l >> part_bits;
    double t1 = none, t2 = none;
    if (g < a.groups)
      for (int i = l & ((1 << part_bits) - 1); i < a.size; i += 1 << part_bits) {
        const int e = g * a.size + i;
        const double x = __builtin_bit_cast(double, (uint64_t)low[e] | (uint64_t)high[e] << 32);
        t2 = fmax(t2, fmin(t1, x));
        t1 = fmax(t1, x);
      }
    for (int o = 1; o < 1 << part_bits; o <<= 1) {
      const double u1 = __shfl_xor(t1, o), u2 = __shfl_xor(t2, o);
      t2 = fmax(fmax(t2, u2), fmin(t1, u1));
      t1 = fmax(t1, u1);
    }
    const double mine = a.best > 1 && t2 > none ? t1 + t2 : t1;
    const uint64_t words = __builtin_bit_cast(uint64_t, mine);
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
      const double x = __builtin_bit_cast(
          double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)words, h << part_bits) |
                      (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(words >> 32), h << part_bits) << 32);
      rank += x > mine || (x == mine && h < g) ? 1 : 0;
    }
    const uint64_t open = __ballot(g < a.groups && rank < a.open && mine > none);
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      const int e = l + 64 * q;
      const uint32_t of = min((uint32_t)e * a.per_size >> 20, (uint32_t)a.groups - 1u);
      if (!(open >> (of << part_bits) & 1u)) v[q] = none;
    }
    if (!a.bias) {                                     // (the logits tell more of what is near 0 or 1)
#pragma unroll
      for (int q = 0; q < PER; ++q)
        if (v[q] > none) v[q] = (double)to_f32(row[l + 64 * q]);
    }
    wave_sync();
  }
  int id = -1;
  for (int j = 0; j < k; ++j) {
    double best = v[0];
#pragma unroll
    for (int q = 1; q < PER; ++q) best = fmax(best, v[q]);
    best = max_wave(best);
    if (!(best > none)) break;                         // (the same in all lanes)
    uint32_t e = 0xFFFFFFFFu;
#pragma unroll
    for (int q = PER - 1; q >= 0; --q) e = v[q] == best ? (uint32_t)(l + 64 * q) : e;
    e = reduce_u32<64>(e, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
    if (l == j) id = (int)e;
#pragma unroll
    for (int q = 0; q < PER; ++q) v[q] = (uint32_t)(l + 64 * q) == e ? none : v[q];
  }
  xj = id >= 0 ? to_f32(row[id]) : 0.0f;
  score = id >= 0 ? score64((double)xj) : 0.0;
  return id;
}

// The whole number below x; 0 for NaN and below 0, -inf among them. (The instruction itself: the language's
// conversion leaves these open, and a bound before it costs an instruction for each value.)
__device__ __forceinline__ uint32_t whole_units(float x) {
  uint32_t u;
  asm("v_cvt_u32_f32 %0, %1" : "=v"(u) : "v"(x));
  return u;
}

// One block of 64 tokens per workgroup, LPR lanes a row, as in route.hip.
template <typename T, int LPR, int VPT, int NT>
__global__ void __launch_bounds__(NT, NT == 512 ? (LPR == 16 ? 4 : 2) : 1)
route_scored_rows_kernel(ScoredArgs a) {
  using L = Lay<T, LPR, VPT>;
  constexpr int AT_ONCE = NT / LPR, WAVES = NT / 64;
  constexpr int BITS = LPR * VPT <= 256 ? 8 : 10;      // of a key, for the expert's number
  constexpr uint32_t LOW = (1u << BITS) - 1u;
  // Two values whose keys differ by more than NEAR are surely in the keys' order. With r the largest |bias|, n
  // the largest score (sigmoid: 1) and m = n + r half the range, a key's unit is m 2^-23 (10 BITS: m 2^-21).
  // The difference of two near values is off by, in m 2^-24,
  //   the sums with the bias: 1 each, 2;
  //   sigmoid: 4 ulp of each score, 8. In all 10, 5 units (1.3);
  //   softmax: 4 (2 ulp) of each exponential, 0.4 n for its argument's rounding (d e^-d), 1 for the product with
  //     1 / sum: 10.8 n of both. And the error of 1 / sum, which they share, times the scores' difference: the
  //     terms' 4 and at most 3.4 (4.5) for their arguments, 19 (21) additions, the division: 27.4 (30.5). That
  //     difference is at most n, and for near values, being their biases', 2 r. 10.8 n + 27.4 min(n, 2 r) is
  //     largest at n = 2 r = 2/3 m: 25.5 (27.5), with the sums 27.5 (29.5), 13.7 units (3.7);
  //   the logits themselves (no bias, no groups): nothing.
  // Forming a key rounds to half a whole number (a quarter) and cuts: 2 units (1.5) for two. `units`, being the
  // same for both, scales their difference alone.
  constexpr uint32_t NEAR = BITS == 8 ? 16 : 8;
  __shared__ uint32_t took[2][MAX_E];
  __shared__ short chosen[ROWS][MAX_K];
  __shared__ float psum[WAVES][LPR * VPT];
  // (the bias is read again for each row: in registers it would not leave room for the rest)
  __shared__ __attribute__((aligned(16))) float bias_of[LPR * VPT];
  __shared__ int count[MAX_E], off[MAX_E + 1];
  __shared__ int wave_sum[WAVES];
  __shared__ int n_routed, n_again;
  // rows that are done again in 64 bits: among all experts, with a NaN
  constexpr int UNSURE = 64, BAD = 128;
  __shared__ short again[ROWS];
  __shared__ short few[ROWS][MAX_K + 1];               // or among these
  __shared__ __attribute__((aligned(8))) float values[AT_ONCE][LPR * VPT];     // where groups are chosen
  __shared__ float group_value[AT_ONCE][MAX_GROUPS];
  __shared__ __attribute__((aligned(16))) uint32_t group_key[AT_ONCE][MAX_GROUPS];
  const int E = a.r.E, k = a.r.k;
  for (int e = threadIdx.x; e < E; e += NT) took[0][e] = took[1][e] = 0u;
  for (int e = threadIdx.x; e < LPR * VPT; e += NT) bias_of[e] = a.bias && e < E ? a.bias[e] : 0.0f;
  if (threadIdx.x == 0) n_routed = n_again = 0;
  // (past the last group: none)
  for (int i = threadIdx.x; i < AT_ONCE * (int)MAX_GROUPS; i += NT) (&group_key[0][0])[i] = 0u;
  __syncthreads();
  const int l = threadIdx.x & (LPR - 1), lane = threadIdx.x & 63;
  const int at_row = threadIdx.x / LPR;
  const int64_t block = (int64_t)a.r.block0 + blockIdx.x;
  const int64_t t0 = block * ROWS;
  const bool by_value = a.bias || a.open < a.groups;
  const bool quads = VPT % 4 == 0 && a.size % 4 == 0;  // (a lane's values lie in fours side by side)
  const int n_quads = a.size / 4;
  uint32_t group_of[(VPT + 3) / 4];                    // of a lane's experts, a byte each
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const uint32_t g = min((uint32_t)L::at(v, l) * a.per_size >> 20, MAX_GROUPS - 1u);
    group_of[v / 4] = (v % 4 ? group_of[v / 4] : 0u) | g << (8 * (v % 4));
  }
  const auto take = [&](int64_t t, int r, int id, float w) __attribute__((always_inline)) {
    a.r.ids[t * k + l] = id;
    a.r.weights[t * k + l] = w;
    chosen[r][l] = (short)id;
    if (id >= 0) atomicOr(&took[r >> 5][id], 1u << (r & 31));
  };
  float acc[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) acc[v] = 0.0f;
  // the range of values, but for what the row adds to it (-inf and NaN close an expert)
  float range = 0.0f;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const float y = bias_of[L::at(v, l)];
    range = __builtin_fmaxf(range, y > -__builtin_inff() ? __builtin_fabsf(y) : 0.0f);
  }
  range = max_lanes<LPR>(range);
  float x[VPT];
  bool on = false;
  const T* row = nullptr;
  const auto fetch = [&](int64_t t) __attribute__((always_inline)) {
    const bool in = t < a.r.T;
    on = in && (!a.r.mask || a.r.mask[t] != 0);
    row = (const T*)a.r.logits + (in ? t : 0) * a.r.ld;
    load_row<T, LPR, VPT>(row, E, l, on, a.r.vec != 0, x);
  };
  fetch(t0 + at_row);
  for (int r0 = 0; r0 < ROWS && t0 + r0 < a.r.T; r0 += AT_ONCE) {
    const int r = r0 + at_row;
    const int64_t t = t0 + r;
    const bool in = t < a.r.T;
    const T* const this_row = row;
    RowSum sum;
    float val[VPT], m, top = -__builtin_inff();        // values (-inf or NaN: never chosen), half their range
    {
      float s[VPT];
      sum = row_scores<LPR, VPT>(x, a.score, s);
      if (by_value) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
          val[v] = x[v] > -__builtin_inff() ? s[v] + bias_of[L::at(v, l)] : -__builtin_inff();
        m = range + (a.score == SCORE_SOFTMAX ? sum.norm : 1.0f);
      } else {
        m = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          val[v] = x[v] + 0.0f;
          m = __builtin_fmaxf(m, x[v] > -__builtin_inff() ? __builtin_fabsf(val[v]) : 0.0f);
        }
        m = max_lanes<LPR>(m);
      }
#pragma unroll
      for (int v = 0; v < VPT; ++v) top = __builtin_fmaxf(top, val[v]);
      top = max_lanes<LPR>(top);
      // (a token that chooses nothing is not in the sums, unless it is NaN)
      const bool bad = sum.share != sum.share;
      const bool little = a.score == SCORE_SIGMOID && top > -__builtin_inff() && !bad &&
                          !(sum.share <= 1.0f / LITTLE && sum.share > 0.0f);
      const float share = (top > -__builtin_inff() && !little) || bad ? sum.share : 0.0f;
#pragma unroll
      for (int v = 0; v < VPT; ++v) acc[v] = __builtin_fmaf(s[v], share, acc[v]);  // (s is NaN in NaN rows alone)
      if (__ballot(little)) {                          // (uniform over the wave)
        float e[VPT], most;
        const float norm = row_softmax<LPR, VPT>(x, most, e);
#pragma unroll
        for (int v = 0; v < VPT; ++v) acc[v] += little ? e[v] * norm : 0.0f;
      }
    }
    // (the next rows' logits are on their way while these choose)
    if (r0 + AT_ONCE < ROWS) fetch(t + AT_ONCE);
    // (no range to count in)
    bool redo = top > -__builtin_inff() && !(m > 1e-30f && m < 1e30f);
    uint32_t open = 0xFFFFFFFFu;
    if (a.open < a.groups) {
      // the values, or where groups are whole quads of experts each quad's two largest
      if (quads) {
        if constexpr (VPT % 4 == 0) {
#pragma unroll
          for (int v = 0; v < VPT; v += 4) {
            float c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = __builtin_fmaxf(val[v + i], -__builtin_inff());       // (NaN)
            const float p = __builtin_fmaxf(c[0], c[1]), q = __builtin_fminf(c[0], c[1]);
            const float u = __builtin_fmaxf(c[2], c[3]), w = __builtin_fminf(c[2], c[3]);
            Pack<float, 2> y;
            y.v[0] = __builtin_fmaxf(p, u);
            y.v[1] = __builtin_fmaxf(__builtin_fminf(p, u), __builtin_fmaxf(q, w));
            *reinterpret_cast<Pack<float, 2>*>(&values[at_row][L::at(v, l) / 2]) = y;
          }
        }
      } else {
#pragma unroll
        for (int v = 0; v < VPT; ++v) values[at_row][L::at(v, l)] = __builtin_fmaxf(val[v], -__builtin_inff());
      }
      wave_sync();
      // 1 << part_bits lanes a group, each with every so manyeth of its values
      const int parts = 1 << a.part_bits, part = l & (parts - 1);
      float least = __builtin_inff(), most = -__builtin_inff();
      uint32_t bits = 0u;
      for (int g0 = 0; g0 < a.groups; g0 += LPR >> a.part_bits) {
        const int g = g0 + (l >> a.part_bits);
        float t1 = -__builtin_inff(), t2 = -__builtin_inff();
        if (g < a.groups) {
          if (quads) {
            const Pack<float, 2>* const from = reinterpret_cast<const Pack<float, 2>*>(&values[at_row][2 * g * n_quads]);
            for (int i = part; i < n_quads; i += parts) {
              const Pack<float, 2> y = from[i];
              t2 = __builtin_fmaxf(__builtin_fmaxf(t2, y.v[1]), __builtin_fminf(t1, y.v[0]));
              t1 = __builtin_fmaxf(t1, y.v[0]);
            }
          } else {
            for (int i = part; i < a.size; i += parts) {
              const float y = values[at_row][g * a.size + i];
              t2 = __builtin_fmaxf(t2, __builtin_fminf(t1, y));
              t1 = __builtin_fmaxf(t1, y);
            }
          }
        }
        for (int o = 1; o < parts; o <<= 1) {
          const float u1 = __shfl_xor(t1, o, LPR), u2 = __shfl_xor(t2, o, LPR);
          t2 = __builtin_fmaxf(__builtin_fmaxf(t2, u2), __builtin_fminf(t1, u1));
          t1 = __builtin_fmaxf(t1, u1);
        }
        const float value = a.best > 1 && t2 > -__builtin_inff() ? t1 + t2 : t1;
        // its order among the groups' values: as a whole number, the lower group first where the five bits
        // that give way to its number decide (nearer than what is done again); 0: nothing to choose
        if (part == 0 && g < a.groups) {
          group_value[at_row][g] = value;
          group_key[at_row][g] = order_key(value) < 32u ? 0u : (order_key(value) & ~31u) | (31u - (uint32_t)g);
        }
      }
      wave_sync();
      // a group's rank among all; the least open and the largest closed value
      for (int g = l; g < a.groups; g += LPR) {
        const uint32_t mine = group_key[at_row][g];
        int rank = 0;
        for (int h = 0; h < a.groups; h += 4) {
          const Pack<uint32_t, 4> y = *reinterpret_cast<const Pack<uint32_t, 4>*>(&group_key[at_row][h]);
#pragma unroll
          for (int i = 0; i < 4; ++i) rank += y.v[i] > mine ? 1 : 0;
        }
        const bool is_open = rank < a.open && mine != 0u;
        const float value = group_value[at_row][g];
        bits |= is_open ? 1u << g : 0u;
        if (is_open) least = __builtin_fminf(least, value);
        else most = __builtin_fmaxf(most, value);
      }
      open = reduce_u32<LPR>(bits, [](uint32_t p, uint32_t q) { return p | q; });
      least = reduce_f32<LPR>(least, [](float p, float q) { return __builtin_fminf(p, q); });
      most = max_lanes<LPR>(most);
      // (two values a side, off as said at NEAR: 4 times 5.4 n, 30.5 min(2 n, 4 r), 4 sums with the bias, and the
      // groups' own sums, up to 2 m, 4: 63 m 2^-24 at most, half of what is asked for. That values alike in the
      // upper bits of their keys went by the group's number shows here as well.)
      redo = redo || (most > -__builtin_inff() && !(least - most > m * 0x1p-17f));
      wave_sync();
    }
    // keys: the value in units of the range's 2^(32 - BITS)th part, from 4 to below all; a -inf gives 0
    // units, and a key below FIRST is never chosen
    constexpr uint32_t FIRST = 1u << BITS;
    const float units = (float)((1u << (31 - BITS)) - 16u) * __builtin_amdgcn_rcpf(__builtin_fmaxf(m, 1e-30f));
    const float least_units = __builtin_fmaf(m, units, 4.0f);
    const uint32_t number = LOW - (uint32_t)L::at(0, l);
    uint32_t key[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      key[v] = (whole_units(__builtin_fmaf(val[v], units, least_units)) << BITS) + number - (uint32_t)L::at(v, 0);
    }
    if (a.open < a.groups) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const uint32_t g = group_of[v / 4] >> (8 * (v % 4)) & 0x1Fu;
        key[v] &= (uint32_t)__builtin_amdgcn_sbfe((int)open, g, 1u);
      }
    }
    // the largest keys one after the other: the next one is the largest below the last, and
    // with d = key - last in wrapping arithmetic every key below it has a larger d than
    // every key from it on
    const auto umax = [](uint32_t p, uint32_t q) { return p > q ? p : q; };
    uint32_t last = 0u, mine = 0u;
    const auto next = [&]() __attribute__((always_inline)) {
      uint32_t d = key[0] - last;
#pragma unroll
      for (int v = 1; v < VPT; ++v) d = umax(d, key[v] - last);
      d = reduce_u32<LPR>(d, umax);
      const uint32_t n = last + d;
      const bool none = n < FIRST || (last != 0u && n >= last);
      last = none ? last : n;
      return none ? 0u : n;
    };
    for (int j = 0; j < k; ++j) {
      const uint32_t n = next();
      if (l == j) mine = n;
    }
    const uint32_t extra = next();
    const int id = mine ? (int)(LOW - (mine & LOW)) : -1;
    const int ie = extra ? (int)(LOW - (extra & LOW)) : -1;
    const float xj = id >= 0 ? to_f32(this_row[id]) : 0.0f;
    const float bj = id >= 0 && a.bias ? a.bias[id] : 0.0f;
    // neighbours among the chosen that are near and not alike; the k-th and the next may be
    // alike and a third near them
    const uint32_t after = (uint32_t)__shfl_down((int)mine, 1, LPR);       // (by all lanes: each gives)
    const uint32_t kn = l == k - 1 ? extra : after;
    const float xn = __shfl_down(xj, 1, LPR), bn = __shfl_down(bj, 1, LPR);
    const bool close = l < k && kn && (mine >> BITS) - (kn >> BITS) <= NEAR && (l == k - 1 || xj != xn || bj != bn);
    const bool near = reduce_u32<LPR>(close ? 1u : 0u, umax) != 0u && !redo;
    bool sure = false;
    if (__ballot(near)) {                              // (uniform over the wave)
      // the choice is among these and the next, if no other expert is near the k-th
      const uint32_t beyond = next(), kth = (uint32_t)__shfl((int)mine, k - 1, LPR);
      sure = near && (beyond == 0u || (kth >> BITS) - (beyond >> BITS) > NEAR);
      if (in && sure && l < k) few[r][l] = (short)id;
      if (in && sure && l == 0) few[r][k] = (short)ie;
    }
    float w = id >= 0 ? score_of(xj, a.score, sum) : 0.0f;
    if (a.r.renorm) w = chosen_share<LPR>(w, xj, id >= 0);
    const bool bad = sum.share != sum.share;
    w = bad ? sum.share : w * a.scale;
    if (in && l < k && !redo && !near) {
      take(t, r, id, w);
      if (l == 0 && id >= 0) atomicAdd(&n_routed, 1);
    }
    if (in && l == 0 && (redo || near)) 
      again[atomicAdd(&n_again, 1)] = (short)(r | (sure ? 0 : UNSURE) | (bad ? BAD : 0));
  }
  __syncthreads();
  // rows whose values are too near: a wave each
  constexpr int PER = (LPR * VPT + 63) / 64;
  const int wave = threadIdx.x >> 6;
  for (int i = wave; i < n_again; i += WAVES) {
    const int r = again[i] & 63;
    const bool sure = (again[i] & UNSURE) == 0, bad = (again[i] & BAD) != 0;
    const int64_t t = t0 + r;
    const T* const row = (const T*)a.r.logits + t * a.r.ld;
    double score;
    float xj;
    const int id = choose64<T, PER>(row, a, lane, sure ? few[r] : nullptr, reinterpret_cast<uint32_t*>(&values[wave * (64 / LPR)][0]),
                                    reinterpret_cast<uint32_t*>(&psum[wave][0]), a.part_bits64, xj, score);
    float w = (float)score;
    if (a.r.renorm) w = chosen_share<64>(w, xj, id >= 0);
    w = bad ? __builtin_nanf("") : w * a.scale;
    if (lane < k) {
      a.r.ids[t * k + lane] = id;
      a.r.weights[t * k + lane] = w;
      chosen[r][lane] = (short)id;
      if (id >= 0) atomicOr(&took[r >> 5][id], 1u << (r & 31));
      if (lane == 0 && id >= 0) atomicAdd(&n_routed, 1);
    }
  }
  finish_block<T, LPR, VPT, NT>(a.r, block, acc, took, chosen, psum, count, off, wave_sum, n_routed);
}

// Workgroups per CU of the backward pass: two where a lane holds much of a row and its factors, which each
// workgroup forms once (2 / 4 / 8: T 32768 E 256 bf16 18.1 / 20.4 / 25.9 us, fp32 18.9 / 19.9 / 21.7,
// T 8192 E 1024 18.5 / 20.3 / 22.0), four where rows are short (T 65536 E 64 14.3 / 12.1 / 11.7).
int bwd_per_cu(int E) { return E > 128 ? 2 : 4; }

struct ScoredBwdArgs {
  const void* logits;
  void* d_logits;
  const int32_t *ids, *counts, *routed;
  const float *dw, *dloss;
  int64_t T, ld, ldd;
  int E, k, renorm, vec, score;
  float coef, scale;
};

// A workgroup walks rows, LPR lanes a row, the scores formed again from the logits. With
// f_e = E c_e / (k n^2) coef dL, shares q = s / sum s and u = s / (the sum of the chosen s), d = scale
// dw, and for the chosen
//   softmax: c = u (d - sum d u) with renormalise, else s d;   dx = q (f - sum f q - [else] sum s d) + c
//   sigmoid: c = u (1 - s) (d - sum d u), else s (1 - s) d;   dx = q (1 - s) (f - sum f q) + c
// which divides by no sum that could be little, and forms 1 - s without cancellation. Vector unit and loads take
// about as long (T 20011 E 160 fp32 10.1 us, 2.5 TB/s; T 32768 E 256 18.9, 3.6 TB/s).
template <typename T, int LPR, int VPT>
__global__ void __launch_bounds__(THREADS)
route_scored_backward_kernel(ScoredBwdArgs a) {
  using L = Lay<T, LPR, VPT>;
  constexpr int AT_ONCE = THREADS / LPR;
  __shared__ __attribute__((aligned(16))) float chosen[AT_ONCE][LPR * VPT];
  const int E = a.E, k = a.k;
  const int l = threadIdx.x & (LPR - 1), group = threadIdx.x / LPR;
  const int n = a.routed[0];
  const float fac = a.dloss && n > 0
                        ? (float)((double)a.dloss[0] * a.coef * E / ((double)k * (double)n * (double)n))
                        : 0.0f;
  float f[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int e = L::at(v, l);
    f[v] = e < E ? fac * (float)a.counts[e] : 0.0f;
  }
  // (a row's loads are issued while the one before it is worked on)
  const int64_t stride = (int64_t)gridDim.x * AT_ONCE;
  int id_n;
  float dw_n, x_n[VPT];
  const auto fetch = [&](int64_t t) __attribute__((always_inline)) {
    const bool in = t < a.T;
    id_n = in && l < k ? a.ids[t * k + l] : -1;
    dw_n = in && l < k && a.dw ? a.dw[t * k + l] : 0.0f;
    load_row<T, LPR, VPT>((const T*)a.logits + (in ? t : 0) * a.ld, E, l, in, a.vec != 0, x_n);
  };
  fetch((int64_t)blockIdx.x * AT_ONCE + group);
  for (int64_t t0 = (int64_t)blockIdx.x * AT_ONCE; t0 < a.T; t0 += stride) {
    const int64_t t = t0 + group;
    const bool in = t < a.T;
    const T* const row = (const T*)a.logits + (in ? t : 0) * a.ld;
    int id = id_n;
    float dwj = dw_n * a.scale;
    float x[VPT], s[VPT], rest[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) x[v] = x_n[v];
    if (t0 + stride < a.T) fetch(t + stride);
    if (id >= E || id < 0) id = -1;
    const float xj = id >= 0 ? to_f32(row[id]) : 0.0f;
    const bool on = __shfl(id, 0, LPR) >= 0;
    float sj, rj = 1.0f, share = 1.0f;
    if (a.score == SCORE_SOFTMAX) {
      float top;
      const float norm = row_softmax<LPR, VPT>(x, top, s);
      sj = exp_neg(xj - top) * norm;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        s[v] *= norm;
        rest[v] = 1.0f;
      }
    } else {
      float z = 0.0f;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        s[v] = sigmoid(x[v], rest[v]);
        z += s[v];
      }
      z = sum_lanes<LPR>(z);
      share = 1.0f / z;
      sj = sigmoid(xj, rj);
      little_scores<LPR, VPT>(x, z < LITTLE, s, share);
    }
    float c = 0.0f, dot = 0.0f;
    if (a.renorm) {
      const float u = chosen_share<LPR>(sj, xj, id >= 0);
      c = u * rj * (dwj - sum_lanes<LPR>(id >= 0 ? dwj * u : 0.0f));
    } else if (id >= 0) {
      c = sj * rj * dwj;
      if (a.score == SCORE_SOFTMAX) dot = c;
    }
    // sum f q [+ sum s d]
#pragma unroll
    for (int v = 0; v < VPT; ++v) dot = __builtin_fmaf(s[v] * share, f[v], dot);
    dot = sum_lanes<LPR>(dot);
    // (a row is its wave's own: LDS accesses of a wave stay in order)
#pragma unroll
    for (int v = 0; v < VPT; ++v) chosen[group][L::at(v, l)] = 0.0f;
    wave_sync();
    if (id >= 0) chosen[group][id] = c;
    wave_sync();
    float g[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      g[v] = s[v] * share * rest[v] * (f[v] - dot) + chosen[group][L::at(v, l)];
    wave_sync();
    if (!in) continue;                                 // (whole rows: no lane of a row is left out)
    T* const out = (T*)a.d_logits + t * a.ldd;
#pragma unroll
    for (int q = 0; q < VPT / L::W; ++q) {
      const int e0 = L::at(q * L::W, l);
      Pack<T, L::W> p;
#pragma unroll
      for (int w = 0; w < L::W; ++w) p.v[w] = from_f32<T>(on ? g[q * L::W + w] : 0.0f);
      if (a.vec != 0 && e0 + L::W <= E) {
        *reinterpret_cast<Pack<T, L::W>*>(out + e0) = p;
      } else {
#pragma unroll
        for (int w = 0; w < L::W; ++w)
          if (e0 + w < E) out[e0 + w] = p.v[w];
      }
    }
  }
}

// The kernels for a type, an E and a number of tokens: as in route.hip, 16 lanes a row up to 256 experts,
// 64 above and for up to four tokens (T 4, E 256 7.8 us; five with 16 lanes 11.2). With 12 values a
// lane and more the workgroups are of 512 threads, two on a CU, which overlaps one's end with the other's
// start (T 32768, E 256 42.5 us, with 1024 51.9; T 20000 37.7 / 41.4; T 32 11.8 / 14.2), but where the
// blocks are no more than the CUs and have two rows for each group of lanes (T 33 16.4 / 14.3, T 4096
// 29.6 / 26.7, T 16384 34.9 / 32.6). Up to 512 experts 64 lanes of 8 values are too few rows at once with 512
// threads (T 65536, E 512 160 us, with 512 193), above them 1024 threads would spill (T 8192, E 1024 82 / 91).
typedef void (*RowsFn)(ScoredArgs);
typedef void (*BwdFn)(ScoredBwdArgs);
struct Pick {
  RowsFn rows;
  int rows_threads;
  BwdFn bwd;
  int rows_at_once, lanes;
};
enum Width { FEW, NARROW, WIDE };                      // 256, 512 or 1024, 1024 threads
template <typename T, Width W>
Pick pick_for(int E) {
#define FP8G_PICK(LPR_, VPT_, NT_)                                                        \
  Pick { route_scored_rows_kernel<T, LPR_, VPT_, NT_>, NT_,                               \
         route_scored_backward_kernel<T, LPR_, VPT_>, THREADS / LPR_, LPR_ }
  constexpr int NT = W == FEW ? THREADS : 1024, MANY = W == WIDE ? 1024 : 512;
  if (E <= 16) return FP8G_PICK(16, 1, NT);
  if (E <= 32) return FP8G_PICK(16, 2, NT);
  if (E <= 64) return FP8G_PICK(16, 4, NT);
  if constexpr (W == FEW) {
    if (E <= 256) return FP8G_PICK(64, 4, NT);
  } else {
    if (E <= 128) return FP8G_PICK(16, 8, NT);
    if (E <= 192) return FP8G_PICK(16, 12, MANY);
    if (E <= 256) return FP8G_PICK(16, 16, MANY);
  }
  if (E <= 512) return FP8G_PICK(64, 8, NT);
  return FP8G_PICK(64, 16, (W == FEW ? THREADS : 512));
#undef FP8G_PICK
}
template <typename T>
Pick pick_of(int E, int64_t tokens, int cus) {
  if (tokens <= 4) return pick_for<T, FEW>(E);
  return tokens > ROWS / 2 && tokens <= (int64_t)ROWS * cus ? pick_for<T, WIDE>(E) : pick_for<T, NARROW>(E);
}
Pick pick(int type, int E, int64_t T, int cus) {
  return type == TYPE_F32    ? pick_of<float>(E, T, cus)
         : type == TYPE_BF16 ? pick_of<bf16_t>(E, T, cus)
                             : pick_of<f16_t>(E, T, cus);
}

}  // namespace

hipError_t launch_route_scored(const ScoredCall& c, hipStream_t stream, int cu_count) {
  ScoredArgs a;
  a.r = route_args(c.route);
  a.bias = c.bias;
  a.score = c.score;
  a.groups = c.groups;
  a.open = c.open;
  a.best = c.best;
  a.size = c.route.E / c.groups;
  a.per_size = (1u << 20) / (uint32_t)a.size + 1u;     // (exact for e below 1024: e size < 2^20)
  a.scale = c.scale;
  const int64_t nblk = (c.route.T + ROWS - 1) / ROWS;
  if (nblk == 0) return launch_route_places(c.route, stream);
  const Pick p = pick(c.route.type, c.route.E, c.route.T, cu_count);
  a.part_bits = a.part_bits64 = 0;
  while (c.groups << (a.part_bits + 1) <= p.lanes) ++a.part_bits;
  while (c.groups << (a.part_bits64 + 1) <= 64) ++a.part_bits64;
  const int64_t most = rows_blocks_max(p.rows_threads);
  for (int64_t b = 0; b < nblk; b += most) {
    a.r.block0 = (int)b;
    const int64_t grid = nblk - b < most ? nblk - b : most;
    p.rows<<<dim3((unsigned)grid), dim3((unsigned)p.rows_threads), 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return nblk > 1 ? launch_route_places(c.route, stream) : hipSuccess;
}

hipError_t launch_route_scored_backward(const ScoredBwdCall& c, hipStream_t stream, int cu_count) {
  const RouteBwdCall& r = c.route;
  ScoredBwdArgs a;
  a.logits = r.logits;
  a.d_logits = r.d_logits;
  a.ids = r.ids;
  a.counts = r.counts;
  a.routed = r.routed;
  a.dw = r.dw;
  a.dloss = r.dloss;
  a.T = r.T;
  a.ld = r.ld;
  a.ldd = r.ldd;
  a.E = r.E;
  a.k = r.k;
  a.renorm = r.renorm;
  a.vec = vec_ok(r.logits, r.ld, r.type) && vec_ok(r.d_logits, r.ldd, r.type);
  a.score = c.score;
  a.coef = r.coef;
  a.scale = c.scale;
  const Pick p = pick(r.type, r.E, r.T, cu_count);
  int64_t grid = (r.T + p.rows_at_once - 1) / p.rows_at_once;
  const int64_t most = (int64_t)cu_count * bwd_per_cu(r.E);
  if (grid > most) grid = most;
  p.bwd<<<dim3((unsigned)grid), dim3(THREADS), 0, stream>>>(a);
  return hipGetLastError();
}

void route_scored_kernels(std::vector<const void*>& out) {
  for (int type : {TYPE_F32, TYPE_BF16, TYPE_F16})
    for (int E : {16, 32, 64, 128, 192, 256, 512, 1024})
      for (int T : {1, 5, 64}) {
        const Pick p = pick(type, E, T, 1);
        out.push_back((const void*)p.rows);
        out.push_back((const void*)p.bwd);
      }
}

}  // namespace fp8g
