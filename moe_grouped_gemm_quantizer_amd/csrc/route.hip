// Routing of tokens to experts: softmax over the experts, the k largest
// logits, the balance loss with its gradient, per-expert counts, and each
// (token, expert) pair's row in the experts' operand.
//
// Mathematics, for a row x of E logits: p = exp(x - max x) / sum exp(x - max x);
// the choice goes by the logits themselves (the softmax is monotone), so it
// does not depend on how p is rounded. Loss: coef sum_e (E c_e / (k n)) (P_e / n)
// with c_e tokens that chose e, n routed tokens, P_e their summed p. Its
// gradient, with the one of the weights, through the softmax's Jacobian:
// dx = p (dp - <p, dp>).
//
// A row's pairs need the number of earlier tokens that chose the same
// expert, over all tokens, so the work has three steps: rows in blocks of 64
// (choice, weights, each block's counts, sums of p, and ranks inside the
// block), a scan of the counts over the blocks, and the final slots. Up to
// 64 tokens are one block, and one launch does everything; small tables of
// counts are scanned by every workgroup of the last step, in two launches.
//
// Measured on the GPU: T 1, E 256, k 8 5.1 us; T 4096, E 8, k 2 4.3 + 4.4 us; T
// 32768, E 256, k 8, fp32 22.2 + 7.2 + 5.3 us where reading the logits takes 6.5,
// bf16 18.1 + 7.2 + 5.2; backward T 30011, E 160, k 6, fp32 13.1 us (38 MB: 7.5 us).

#include <vector>

#include "route_common.h"

namespace fp8g {
namespace {

// One block of 64 tokens per workgroup; LPR lanes per row. With 1024 threads
// (16 lanes per row) all rows of a block are worked on at once: its time is
// that of one row's chain of dependent steps, which four waves that walk the
// block go through four times (T 4096, E 8: 6.4 -> 4.5 us; T 32768, E 256: 27
// -> 26). Bound by the vector unit at many experts: about 990 instructions for
// four rows of 256, 13 us of the 22 at T 32768, after the loads (6.5), which a
// workgroup's two sets of rows do not overlap with them.
template <typename T, int LPR, int VPT, int NT>
__global__ void __launch_bounds__(NT)
route_rows_kernel(RouteArgs a) {
  constexpr int AT_ONCE = NT / LPR;
  constexpr int WAVES = NT / 64;
  __shared__ uint32_t took[2][MAX_E];                  // tokens of the block that chose e, as bits
  __shared__ short chosen[ROWS][MAX_K];
  __shared__ float psum[WAVES][LPR * VPT];
  __shared__ int count[MAX_E], off[MAX_E + 1];         // (where one block is all)
  __shared__ int wave_sum[WAVES];
  __shared__ int n_routed;
  const int E = a.E, k = a.k;
  for (int e = threadIdx.x; e < E; e += NT) took[0][e] = took[1][e] = 0u;
  if (threadIdx.x == 0) n_routed = 0;
  __syncthreads();
  const int l = threadIdx.x & (LPR - 1);
  const int64_t block = (int64_t)a.block0 + blockIdx.x;
  const int64_t t0 = block * ROWS;
  float acc[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) acc[v] = 0.0f;
  for (int r0 = 0; r0 < ROWS && t0 + r0 < a.T; r0 += AT_ONCE) {
    const int r = r0 + (int)threadIdx.x / LPR;
    const int64_t t = t0 + r;
    const bool in = t < a.T;
    const bool on = in && (!a.mask || a.mask[t] != 0);
    float x[VPT], ex[VPT];
    load_row<T, LPR, VPT>((const T*)a.logits + (in ? t : 0) * a.ld, E, l, on, a.vec != 0, x);
    float top;
    const float inv = row_softmax<LPR, VPT>(x, top, ex);
#pragma unroll
    for (int v = 0; v < VPT; ++v) acc[v] += ex[v] * inv;
    float xj;
    const int id = choose<T, LPR, VPT>(x, (const T*)a.logits + (in ? t : 0) * a.ld, l, k, xj);
    float w = id >= 0 ? exp_neg(xj - top) : 0.0f;
    const float s = a.renorm ? sum_lanes<LPR>(w) : 0.0f;
    // (a NaN row: inv is NaN, and so is every weight)
    w = inv != inv ? inv : (a.renorm ? (s > 0.0f ? w / s : 0.0f) : w * inv);
    if (in && l < k) {
      a.ids[t * k + l] = id;
      a.weights[t * k + l] = w;
      chosen[r][l] = (short)id;
      if (id >= 0) {
        atomicOr(&took[r >> 5][id], 1u << (r & 31));
        if (l == 0) atomicAdd(&n_routed, 1);
      }
    }
  }
  finish_block<T, LPR, VPT, NT>(a, block, acc, took, chosen, psum, count, off, wave_sum, n_routed);
}

// Scan over the blocks, 16 experts per workgroup, 64 runs of blocks side by
// side: counts become the tokens of earlier blocks (in place), the totals go
// out. The last column holds the routed tokens.
constexpr int RUNS = 64, COLS = 16;
__global__ void __launch_bounds__(COLS * RUNS)
route_scan_kernel(RouteArgs a, int nblk) {
  __shared__ int cnt[RUNS][COLS];
  __shared__ double prob[RUNS][COLS];
  const int l = threadIdx.x % COLS, run = threadIdx.x / COLS;
  const int e = blockIdx.x * COLS + l;
  const int E = a.E;
  const int per = (nblk + RUNS - 1) / RUNS;
  const int b0 = min(nblk, run * per), b1 = min(nblk, b0 + per);
  // (loads in batches: a run is a chain of them otherwise)
  constexpr int BATCH = 8;
  int s = 0;
  double p = 0.0;
  if (e <= E) {
    for (int b = b0; b < b1; b += BATCH) {
      int c[BATCH];
      float q[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int64_t at = min(b + i, b1 - 1);
        c[i] = a.part_count[at * (E + 1) + e];
        q[i] = e < E ? a.part_prob[at * E + e] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        s += b + i < b1 ? c[i] : 0;
        p += b + i < b1 ? (double)q[i] : 0.0;
      }
    }
  }
  cnt[run][l] = s;
  prob[run][l] = p;
  __syncthreads();
  if (e > E) return;
  int at = 0;
  for (int q = 0; q < run; ++q) at += cnt[q][l];
  for (int b = b0; b < b1; b += BATCH) {
    int c[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) c[i] = a.part_count[(int64_t)min(b + i, b1 - 1) * (E + 1) + e];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (b + i < b1) {
        a.part_count[(int64_t)(b + i) * (E + 1) + e] = at;
        at += c[i];
      }
  }
  if (run == RUNS - 1) {
    if (e == E) {
      a.routed[0] = at;
    } else {
      a.counts[e] = at;
      double ps = 0.0;
      for (int q = 0; q < RUNS; ++q) ps += prob[q][l];
      a.prob_sum[e] = (float)ps;
    }
  }
}

// Slots from the ranks; the first workgroup also writes offsets and loss.
constexpr int PAIRS = 4 * THREADS;                     // pairs per workgroup
__global__ void __launch_bounds__(THREADS)
route_slots_kernel(RouteArgs a) {
  __shared__ int off[MAX_E + 1];
  __shared__ int wave_sum[THREADS / 64];
  const int E = a.E, k = a.k;
  // the pairs' loads first: the offsets are formed while they are on their way
  constexpr int Q = PAIRS / THREADS;
  const int64_t pairs = a.T * k;
  const int64_t i0 = (int64_t)blockIdx.x * PAIRS + threadIdx.x;
  int id[Q], rank[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int64_t i = i0 + q * THREADS;
    id[q] = i < pairs ? a.ids[i] : -1;
    rank[q] = i < pairs ? a.slots[i] : 0;
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int64_t blk = (i0 + q * THREADS) / ((int64_t)ROWS * k);
    if (id[q] >= 0) rank[q] += a.part_count[blk * (E + 1) + id[q]];
  }
  if (a.max_m == 0) offsets_of<THREADS>(a.counts, E, a.align, off, wave_sum);
#pragma unroll
  for (int q = 0; q < Q; ++q)                          // (without an expert: the slot is -1 already)
    if (id[q] >= 0) a.slots[i0 + q * THREADS] = slot_of(a, id[q], a.max_m == 0 ? off[id[q]] : 0, rank[q]);
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e <= E; e += THREADS)
      a.offsets[e] = a.max_m == 0 ? off[e] : (int)(e * a.max_m);
    if (threadIdx.x < 64) write_loss(a.counts, a.prob_sum, a.routed[0], E, k, a.coef, a.loss);
  }
}

// Scan and slots in one launch, for tables of counts so small that every
// workgroup may read all of it: one workgroup per block of tokens, EP threads
// (a power of two over E) side by side in a row of the table. Every workgroup
// reads blocks x EP / THREADS entries a thread, so that product decides (scan and slots
// against the joined launch, whole calls): 4096: E 15 13.9 / 12.8 us, E 63 14.8 / 13.0,
// E 255 21.5 / 19.3; 5120: E 8 14.5 / 14.3, E 31 14.5 / 13.7, E 127 16.6 / 16.4; 6144: E 15
// 15.6 / 15.8, E 63 14.5 / 15.6, E 255 21.4 / 22.1; 16384: E 255 22.3 / 33.2.
constexpr int JOIN_MAX = 5120;
__global__ void __launch_bounds__(THREADS)
route_join_kernel(RouteArgs a, int nblk, int EP) {
  __shared__ int before[THREADS], total[THREADS];
  __shared__ int off[MAX_E + 1];
  __shared__ int wave_sum[THREADS / 64];
  __shared__ double prob[THREADS];
  __shared__ float psum[THREADS];
  const int E = a.E, k = a.k, blk = blockIdx.x;
  const int t = threadIdx.x, e = t & (EP - 1), run = t / EP, runs = THREADS / EP;
  const int64_t t0 = (int64_t)blk * ROWS;
  const int pairs = (int)(min((int64_t)ROWS, a.T - t0) * k);
  constexpr int Q = ROWS * MAX_K / THREADS;
  int id[Q], rank[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int i = t + q * THREADS;
    id[q] = i < pairs ? a.ids[t0 * k + i] : -1;
    rank[q] = i < pairs ? a.slots[t0 * k + i] : 0;
  }
  before[t] = total[t] = 0;
  __syncthreads();
  int all = 0, early = 0;
  double p = 0.0;
  if (e <= E) {
#pragma unroll 4
    for (int b = run; b < nblk; b += runs) {
      const int c = a.part_count[(int64_t)b * (E + 1) + e];
      all += c;
      early += b < blk ? c : 0;
      if (blk == 0 && e < E) p += (double)a.part_prob[(int64_t)b * E + e];
    }
    atomicAdd(&total[e], all);
    atomicAdd(&before[e], early);
  }
  prob[t] = p;
  __syncthreads();
  if (a.max_m == 0) offsets_of<THREADS>(total, E, a.align, off, wave_sum);
#pragma unroll
  for (int q = 0; q < Q; ++q)
    if (id[q] >= 0)
      a.slots[t0 * k + t + q * THREADS] =
          slot_of(a, id[q], a.max_m == 0 ? off[id[q]] : 0, before[id[q]] + rank[q]);
  if (blk == 0) {
    if (t <= E) a.offsets[t] = a.max_m == 0 ? off[t] : (int)(t * a.max_m);
    if (t < E) {
      double s = 0.0;
      for (int r = 0; r < runs; ++r) s += prob[r * EP + t];
      a.counts[t] = total[t];
      a.prob_sum[t] = psum[t] = (float)s;
    }
    if (t == 0) a.routed[0] = total[E];
    __syncthreads();
    if (t < 64) write_loss(total, psum, total[E], E, k, a.coef, a.loss);
  }
}

__global__ void route_empty_kernel(RouteArgs a) {
  for (int e = threadIdx.x; e <= a.E; e += THREADS) {
    if (e < a.E) {
      a.counts[e] = 0;
      a.prob_sum[e] = 0.0f;
    }
    a.offsets[e] = (int)(e * a.max_m);
  }
  if (threadIdx.x == 0) {
    a.routed[0] = 0;
    a.loss[0] = 0.0f;
  }
}

// workgroups per CU of the backward pass (T 30011, E 160, fp32: 8: 16.5 us, 6: 13.9, 4: 13.4,
// 2: 14.3; with 8 every workgroup has one set of rows and nothing to load ahead. T 65536,
// E 64, bf16: 11.6, 11.5, 12.2, 15.2)
constexpr int BWD_PER_CU = 4;

struct RouteBwdArgs {
  const void* logits;
  void* d_logits;
  const int32_t *ids, *counts, *routed;
  const float *dw, *dloss;
  int64_t T, ld, ldd;
  int E, k, renorm, vec;
  float coef;
};

// A workgroup walks rows; LPR lanes per row, the softmax computed again from
// the logits (it is cheaper to form than to store and read).
template <typename T, int LPR, int VPT>
__global__ void __launch_bounds__(THREADS)
route_backward_kernel(RouteBwdArgs a) {
  using L = Lay<T, LPR, VPT>;
  // the chosen experts' gradients of each row, in the lanes' order of experts
  constexpr int AT_ONCE = THREADS / LPR;
  __shared__ __attribute__((aligned(16))) float chosen[AT_ONCE][LPR * VPT];
  const int E = a.E, k = a.k;
  const int l = threadIdx.x & (LPR - 1), group = threadIdx.x / LPR;
  const int n = a.routed[0];
  const float fac =
      a.dloss && n > 0
          ? (float)((double)a.dloss[0] * a.coef * E / ((double)k * (double)n * (double)n))
          : 0.0f;
  float f[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int e = L::at(v, l);
    f[v] = e < E ? fac * (float)a.counts[e] : 0.0f;
  }
  // (a row's loads are issued while the one before it is worked on; what a row
  // that takes no part holds does not matter)
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
    const T* row = (const T*)a.logits + (in ? t : 0) * a.ld;
    int id = id_n;
    float dwj = dw_n;
    float x[VPT], ex[VPT], top;
#pragma unroll
    for (int v = 0; v < VPT; ++v) x[v] = x_n[v];
    if (t0 + stride < a.T) fetch(t + stride);
    if (id >= E || id < 0) id = -1;
    const float xj = id >= 0 ? to_f32(row[id]) : 0.0f;
    const bool on = __shfl(id, 0, LPR) >= 0;
    const float inv = row_softmax<LPR, VPT>(x, top, ex);
    const float pj = id >= 0 ? exp_neg(xj - top) * inv : 0.0f;
    if (id < 0) dwj = 0.0f;
    if (a.renorm) {
      const float s = sum_lanes<LPR>(pj);
      const float c = sum_lanes<LPR>(id >= 0 ? dwj * pj : 0.0f);
      dwj = id >= 0 && !(s <= 0.0f) ? (dwj - c / s) / s : 0.0f;
    }
    float dot = id >= 0 ? pj * dwj : 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      ex[v] *= inv;
      dot = __builtin_fmaf(ex[v], f[v], dot);
    }
    dot = sum_lanes<LPR>(dot);
    // (a row is its wave's own: LDS accesses of a wave stay in order)
    float g[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) chosen[group][L::at(v, l)] = 0.0f;
    wave_sync();
    if (id >= 0) chosen[group][id] = dwj;
    wave_sync();
#pragma unroll
    for (int v = 0; v < VPT; ++v) g[v] = f[v] - dot + chosen[group][L::at(v, l)];
    wave_sync();
    if (!in) continue;                                 // (whole rows: no lane of a row is left out)
    T* out = (T*)a.d_logits + t * a.ldd;
#pragma unroll
    for (int q = 0; q < VPT / L::W; ++q) {
      const int e0 = L::at(q * L::W, l);
      Pack<T, L::W> p;
#pragma unroll
      for (int w = 0; w < L::W; ++w) {
        const int v = q * L::W + w;
        p.v[w] = from_f32<T>(on ? ex[v] * g[v] : 0.0f);
      }
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

// The kernels for a type and an E: 16 lanes per row up to 256 experts (a DPP
// row: reductions take four steps, and four rows share every instruction), 64
// above; and 64 for the rows of up to four tokens, where a row's latency counts
// (T 1, E 256, k 8).
typedef void (*RowsFn)(RouteArgs);
typedef void (*BwdFn)(RouteBwdArgs);
struct Pick {
  RowsFn rows;
  int rows_threads;
  BwdFn bwd;
  int rows_at_once;
};
template <typename T, int NT>
Pick pick_for(int E) {
  constexpr bool few = NT == THREADS;
  // (from 12 values a lane on, two workgroups of 512 threads fit a CU's registers
  // and one of 1024 alone: T 32768, fp32, E 256 23.5 -> 22.1 us, E 160 18.9 -> 17.2; whole
  // calls of E 64 19.7 -> 20.3)
  constexpr int WIDE = NT > 512 ? 512 : NT;
#define FP8G_PICK(LPR_, VPT_)                                                             \
  Pick { route_rows_kernel<T, LPR_, VPT_, LPR_ == 16 && VPT_ >= 12 ? WIDE : NT>,          \
         LPR_ == 16 && VPT_ >= 12 ? WIDE : NT, route_backward_kernel<T, LPR_, VPT_>,      \
         THREADS / LPR_ }
  if (E <= 16) return FP8G_PICK(16, 1);
  if (E <= 32) return FP8G_PICK(16, 2);
  if (E <= 64) return FP8G_PICK(16, 4);
  if constexpr (few) {
    if (E <= 256) return FP8G_PICK(64, 4);
  } else {
    if (E <= 128) return FP8G_PICK(16, 8);
    if (E <= 192) return FP8G_PICK(16, 12);
    if (E <= 256) return FP8G_PICK(16, 16);
  }
  if (E <= 512) return FP8G_PICK(64, 8);
  return FP8G_PICK(64, 16);
#undef FP8G_PICK
}
template <typename T>
Pick pick_of(int E, int64_t tokens) {
  return tokens <= 4 ? pick_for<T, THREADS>(E) : pick_for<T, 1024>(E);
}
Pick pick(int type, int E, int64_t T) {
  return type == TYPE_F32    ? pick_of<float>(E, T)
         : type == TYPE_BF16 ? pick_of<bf16_t>(E, T)
                             : pick_of<f16_t>(E, T);
}

}  // namespace

int64_t route_blocks(int64_t T) { return (T + ROWS - 1) / ROWS; }

size_t route_workspace_bytes(int64_t T, int E) {
  const int64_t nblk = route_blocks(T);
  if (nblk <= 1) return 0;
  return ((size_t)nblk * (E + 1) * sizeof(int) + 15) / 16 * 16 + (size_t)nblk * E * sizeof(float);
}

hipError_t launch_route_places(const RouteCall& c, hipStream_t stream) {
  const RouteArgs a = route_args(c);
  const int64_t nblk = route_blocks(c.T);
  if (nblk == 0) {
    route_empty_kernel<<<dim3(1), dim3(THREADS), 0, stream>>>(a);
    return hipGetLastError();
  }
  int ep = 1;
  while (ep <= c.E) ep *= 2;
  if (nblk > 1 && ep <= THREADS && nblk * ep <= JOIN_MAX) {
    route_join_kernel<<<dim3((unsigned)nblk), dim3(THREADS), 0, stream>>>(a, (int)nblk, ep);
  } else if (nblk > 1) {
    route_scan_kernel<<<dim3((unsigned)(c.E / COLS + 1)), dim3(COLS * RUNS), 0, stream>>>(a, (int)nblk);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t grid = (c.T * c.k + PAIRS - 1) / PAIRS;
    route_slots_kernel<<<dim3((unsigned)grid), dim3(THREADS), 0, stream>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_route(const RouteCall& c, hipStream_t stream) {
  RouteArgs a = route_args(c);
  const int64_t nblk = route_blocks(c.T);
  if (nblk == 0) return launch_route_places(c, stream);
  const Pick p = pick(c.type, c.E, c.T);
  // A launch holds fewer than 2^32 threads (from 2^28 tokens on the rows take several).
  // The kernels after it read what it wrote, places in tables among it: none is launched
  // behind one that was not.
  const int64_t most = rows_blocks_max(p.rows_threads);
  for (int64_t b = 0; b < nblk; b += most) {
    a.block0 = (int)b;
    const int64_t grid = nblk - b < most ? nblk - b : most;
    p.rows<<<dim3((unsigned)grid), dim3((unsigned)p.rows_threads), 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return nblk > 1 ? launch_route_places(c, stream) : hipSuccess;
}

hipError_t launch_route_backward(const RouteBwdCall& c, hipStream_t stream, int cu_count) {
  RouteBwdArgs a;
  a.logits = c.logits;
  a.d_logits = c.d_logits;
  a.ids = c.ids;
  a.counts = c.counts;
  a.routed = c.routed;
  a.dw = c.dw;
  a.dloss = c.dloss;
  a.T = c.T;
  a.ld = c.ld;
  a.ldd = c.ldd;
  a.E = c.E;
  a.k = c.k;
  a.renorm = c.renorm;
  a.vec = vec_ok(c.logits, c.ld, c.type) && vec_ok(c.d_logits, c.ldd, c.type);
  a.coef = c.coef;
  const Pick p = pick(c.type, c.E, c.T);
  int64_t grid = (c.T + p.rows_at_once - 1) / p.rows_at_once;
  if (grid > (int64_t)cu_count * BWD_PER_CU) grid = (int64_t)cu_count * BWD_PER_CU;
  p.bwd<<<dim3((unsigned)grid), dim3(THREADS), 0, stream>>>(a);
  return hipGetLastError();
}

void route_kernels(std::vector<const void*>& out) {
  for (int type : {TYPE_F32, TYPE_BF16, TYPE_F16})
    for (int E : {16, 32, 64, 128, 192, 256, 512, 1024})
      for (int T : {1, 64}) {
        const Pick p = pick(type, E, T);
        out.push_back((const void*)p.rows);
        out.push_back((const void*)p.bwd);
      }
  out.push_back((const void*)route_scan_kernel);
  out.push_back((const void*)route_slots_kernel);
  out.push_back((const void*)route_join_kernel);
  out.push_back((const void*)route_empty_kernel);
}

}  // namespace fp8g
