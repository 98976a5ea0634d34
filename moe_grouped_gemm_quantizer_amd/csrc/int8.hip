// Products in 8-bit integers: the quantiser (one scale a row) and the product with a
// scale for each token and each output channel, dense and for every expert of a layer.
//
// d[m][n] = bf16( (fl32(sum_k a[m][k] b[n][k]) sa[m]) sb[n] ). The sum is a whole number,
// exact in 32 bits up to K = 131071 (codes -128 .. 127: K 2^14 < 2^31), so its order does
// not matter and every way of cutting the work gives the same bits.

#include <type_traits>
#include <vector>

#include "elem.h"
#include "gemm_index.h"
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
// An HBM stream: 4096 x 7168 bf16 in 18.1 us, 4.9 TB/s (a large copy: 5.0). A wave a row up to
// 256 pieces, which spares short rows the workgroup's barrier (4096 x 512 bf16 3.4 us, a workgroup a
// row 6.3; 8192 x 2048 12.4 / 12.5), and a workgroup above (4096 x 4096 11.2, a wave with 16 pieces a
// lane 15.4); rows of up to 2048 pieces stay in registers (2048 x 16384 bf16 21.4 us, read twice 27.2).
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
// The product. Codes go from global memory straight into LDS; each 128-byte LDS row holds
// 128 bytes of K of one row, its 16-byte chunks swizzled (swz).

typedef __attribute__((address_space(3))) void* lds_ptr_t;
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_ptr_t)p);
}
// Direct global -> LDS copies, through inline assembly so that the compiler does not wait
// for all of them before the next LDS read; the waits are explicit, before the barrier that
// publishes a stage.
__device__ __forceinline__ void copy16(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "{m0}"(lds)
               : "memory");
}
constexpr int vmcnt_only(int n) { return (n & 0xF) | (0x7 << 4) | (0xF << 8) | (((n >> 4) & 3) << 14); }

// Chunk swizzle of an LDS row of 128 bytes (16-byte chunks): fragment reads of 8 or 16
// consecutive rows meet every bank group equally.
__device__ __forceinline__ int swz(int row, int chunk) { return chunk ^ (row & 7) ^ ((row >> 3) & 1); }

// Fragment f of a band of rows, bytes 64 kh .. +63 of K: lane l holds position l % 32 and 32
// of those bytes, chunks 4 kh + 2 (l / 32) and the next: two operands of the matrix
// instruction (which bytes of K meet in which of them is free, as long as a and b agree).
struct Frag {
  v4i lo, hi;
};
__device__ __forceinline__ Frag read_frag(const uint8_t* band, int f, int kh, int lane) {
  const int r = f * 32 + (lane & 31), c = kh * 4 + (lane >> 5) * 2;
  Frag v;
  v.lo = *reinterpret_cast<const v4i*>(band + r * 128 + swz(r, c) * 16);
  v.hi = *reinterpret_cast<const v4i*>(band + r * 128 + swz(r, c + 1) * 16);
  return v;
}

__device__ __forceinline__ uint32_t bf16_pair(float x, float y) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
}

constexpr int MAX_G = 1024;

// The experts that have rows: first row, rows, and row blocks of those before.
struct Experts {
  int id[MAX_G], row0[MAX_G], rows[MAX_G], before[MAX_G + 1];
  int n;
};

// By one wave; `side`: rows of a block.
__device__ __forceinline__ void list_experts(const Int8Args& a, Experts& ex, int side, int lane) {
  const int R = (int)a.rows;
  int n = 0, blocks = 0, past = 0;                     // past: where the experts before end at the latest
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    const int g = g0 + lane;
    int lo = 0, cnt = 0;
    if (a.mode == MODE_CONTIGUOUS) {
      // an offset below an earlier one counts as that one: no row has two experts, whatever they are
      lo = g < a.G ? min(max(a.group[g], past), R) : 0;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) lo = max(lo, __shfl_up(lo, o));
      const int hi = g < a.G ? min(max(a.group[g + 1], lo), R) : lo;
      cnt = hi - lo;
      past = __shfl(hi, 63);
    } else if (g < a.G) {
      cnt = a.mode == MODE_DENSE ? R : min(max(a.group[g], 0), R);
    }
    const uint64_t has = __ballot(cnt > 0);
    const int i = n + __popcll(has & ((1ull << lane) - 1));
    int sum = (int)(((unsigned)cnt + side - 1) / side);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(sum, o);
      if (lane >= o) sum += y;
    }
    if (cnt > 0) {
      ex.id[i] = g;
      ex.row0[i] = lo;
      ex.rows[i] = cnt;
      ex.before[i + 1] = blocks + sum;
    }
    n += __popcll(has);
    blocks += __shfl(sum, 63);
  }
  if (lane == 0) {
    ex.n = n;
    ex.before[0] = 0;
  }
}

// 256x256 tiles, bound by the matrix unit and, beside it, the issue of its copies and the clock that the
// chip holds under it: 4096x8192x8192 in 210 to 230 us, 2.4 to 2.6 POPS (the library's own product 231 us;
// 128x128 tiles of one workgroup each 319, 256x128 267). Where each weight is read for one row
// block, HBM: 32 experts 7168x2048 of up to 256 rows 112 to 116 us and 32 for the last round, 3.8 TB/s.
// Four waves of 128x128, one per SIMD, the 256 accumulators of a lane in the
// accumulation registers. A workgroup walks tiles (expert, row block, column block); the
// 128-byte steps of all its tiles form one sequence with two LDS stages. A step's 64
// matrix instructions (32 pairs):
//   pairs 0-15   fragments 0 and 1 of b against all of a. After the first four everyone meets:
//          a's part of this stage and b's first half have been read by all (a step ahead),
//          so that the copies of the step after next may go there, and b's second half has
//          landed and is read.
//   pairs 16-31  everyone meets again: this stage is read altogether, and the next one's a and
//          b first half have landed. Each fragment of a against 2 and 3 of b, after which
//          the next step's fragment takes its place.
// Which global row lies in which LDS row is free, as each lane of a copy has its own
// address. The rows of a 128-row band are dealt so that position r of fragment i of a is
// row 4 r + i, and position x of fragment j of b column 4 col_of(x) + j: a lane then ends up
// with runs of 8 adjacent columns of a row (see the store).
constexpr int TS = 256;                                // tile side
constexpr int STAGE = 2 * TS * 128;                    // codes of a and b
constexpr int COPIES = 16;                             // a wave's copies of a stage
constexpr int EARLY = 12;                              // those that are read a step ahead,
constexpr int EARLY_FIRST = 8;                         // of these, issued in a step's first half
constexpr int STORES = 32;                             // a wave's stores of a full tile

// Of `tiles` on `round` workgroups those that are walked whole: all, but for a last round that would
// leave half of the workgroups or more without one. Its tiles go to int8_rest_kernel in two or four
// parts, which take 0.6 of a round as halves, 0.35 as quarters (4096x6144x7168, 1.5 rounds, 195 -> 159
// us; 4096x4608x7168, 1.1, 171 -> 127; 4096 rows over 8 experts, 1.2, 174 -> 139; where weights from
// memory bound the launch, as 8192x7168x2048 with 3.5, 147 -> 149).
__host__ __device__ __forceinline__ uint32_t full_rounds(uint32_t tiles, uint32_t round) {
  const uint32_t rest = tiles % round;
  return rest <= round / 2 ? tiles - rest : tiles;
}

struct Tile {
  const int8_t *a, *b;                                 // first row
  const float *sa, *sb;
  uint16_t* d;
  int mv, nv;                                          // rows and columns that exist
};

__device__ __forceinline__ void tile_of(const Int8Args& a, const Experts& ex, int slot, int nblocks, Tile& t) {
  // the expert whose row blocks hold this tile (all of an expert's tiles in a row)
  int lo = 0, hi = __builtin_amdgcn_readfirstlane(ex.n) - 1;
  const int blk = slot / nblocks;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (blk < __builtin_amdgcn_readfirstlane(ex.before[mid + 1])) hi = mid;
    else lo = mid + 1;
  }
  const int before = __builtin_amdgcn_readfirstlane(ex.before[lo]);
  const int mblocks = __builtin_amdgcn_readfirstlane(ex.before[lo + 1]) - before;
  int mb, nb;
  gidx::swizzle_tile(slot - before * nblocks, mblocks, nblocks, 4, mb, nb);
  const int64_t g = __builtin_amdgcn_readfirstlane(ex.id[lo]);
  const int64_t m0 = (int64_t)mb * TS, n0 = (int64_t)nb * TS;
  const int rows = __builtin_amdgcn_readfirstlane(ex.rows[lo]);
  const int64_t row = (a.mode == MODE_MASKED ? g * a.rows : __builtin_amdgcn_readfirstlane(ex.row0[lo])) + m0;
  t.mv = (int)min((int64_t)TS, rows - m0);
  t.nv = (int)min((int64_t)TS, a.N - n0);
  t.a = a.a + row * a.K;
  t.sa = a.sa + row;
  t.b = a.b + (g * a.N + n0) * a.K;
  t.sb = a.sb + g * a.N + n0;
  t.d = a.d + row * a.N + n0;
}

// This lane's copy offsets for a tile. Wave w copies the LDS rows of band w / 2 whose bit 3 is
// w % 2: copy c of an operand is fragment c % 4, positions 16 (c / 4) + 8 (w % 2) .. +7. Rows
// past the tile's last are copies of it (read in bounds, never stored).
struct Plan {
  uint32_t va, ma, vb, mb;                             // copy 0's offset, the last row's
};
__device__ __forceinline__ int col_of(int x) {         // position of b -> column / 4
  return (x & 1) | ((x >> 2) & 1) << 1 | ((x >> 1) & 1) << 2 | (x >> 3) << 3;
}
__device__ __forceinline__ void make_plan(Plan& p, const Int8Args& a, const Tile& t, int wave, int lane) {
  const int band = wave >> 1, h = wave & 1, r = h * 8 + (lane >> 3);
  const uint32_t ch = (uint32_t)((lane & 7) ^ (lane >> 3) ^ h) * 16u, K = (uint32_t)a.K;
  p.va = (uint32_t)(band * 128 + r * 4) * K + ch;
  p.vb = (uint32_t)(band * 128 + col_of(r) * 4) * K + ch;
  p.ma = (uint32_t)(t.mv - 1) * K + ch;
  p.mb = (uint32_t)(t.nv - 1) * K + ch;
}

// Copy c of a wave's share of a stage: a's eight, b's fragments 0 and 1, b's 2 and 3.
__device__ __forceinline__ void issue(const Plan& p, const Int8Args& a, const Tile& t, int kb, uint32_t stage,
                                      int wave, int c) {
  const uint32_t dst = stage + (uint32_t)((wave >> 1) * 16 + (wave & 1)) * 1024u;
  // (opaque: formed at each copy, the 16 offsets would otherwise be kept in registers that
  // the fragments need)
  uint32_t K = (uint32_t)a.K;
  asm volatile("" : "+s"(K));
  if (c < 8) {
    const int f = c & 3, half = c >> 2;
    copy16(t.a + (int64_t)kb * 128, min(p.va + (uint32_t)(f + 64 * half) * K, p.ma),
           dst + (uint32_t)(f * 4096 + half * 2048));
  } else {
    const int q = c - 8, f = q >> 1, half = q & 1;
    copy16(t.b + (int64_t)kb * 128, min(p.vb + (uint32_t)(f + 64 * half) * K, p.mb),
           dst + TS * 128 + (uint32_t)(f * 4096 + half * 2048));
  }
}

// K is a multiple of 128 here. Where it is not, each copy touches two 128-byte lines for one, and
// this kernel, bound by its copies, fell behind the smaller tiles (4644x12112x7904 775 against
// 612 us, 1128x7184x4016 112 / 76), so it is not built for that.
__global__ void __launch_bounds__(256, 1)
int8_tile_kernel(Int8Args a, int nblocks, int xcd_remap) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STAGE];
  __shared__ Experts ex;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grid = gridDim.x, w = blockIdx.x;
  if (wave == 0) list_experts(a, ex, TS, lane);
  __syncthreads();
  const int n_ex = __builtin_amdgcn_readfirstlane(ex.n);
  const int tiles = (int)full_rounds(__builtin_amdgcn_readfirstlane(ex.before[n_ex]) * nblocks, a.round);
  const int first = xcd_remap ? (w & 7) * (grid >> 3) + (w >> 3) : w;
  if (first >= tiles) return;
  const int steps = (int)(a.K / 128);
  const int wm = wave >> 1, wn = wave & 1;
  const uint32_t base = lds_addr(lds);
  // copy cursor
  int p_slot = first, p_kb = 0;
  Tile tp;
  tile_of(a, ex, p_slot, nblocks, tp);
  Plan pl;
  make_plan(pl, a, tp, wave, lane);
  auto advance = [&]() __attribute__((always_inline)) {
    // (past the last step it stays there: two stages are copied once more at the end, for
    // nothing, and every wait may count on the same copies)
    if (++p_kb == steps) {
      if (p_slot + grid < tiles) {
        p_kb = 0;
        p_slot += grid;
        tile_of(a, ex, p_slot, nblocks, tp);
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
  v16i acc[4][4];
  Frag af[4][2], bf[4][2];       // fragments of a and b, by halves of the 128 bytes
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

  // Two points of a step where everyone waits for copies and meets: for b's late fragments of
  // this step, and half way for the early part of the next. N copies have been issued since
  // those; for three points after a full tile its stores are newer too. (Waits may be longer
  // than needed, never shorter: where a ragged tile stores less, its stores are waited for.)
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
    tile_of(a, ex, slot, nblocks, tc);
    // (a tile's first step starts its sums from a zero operand)
    auto step = [&](auto first_step) __attribute__((always_inline)) {
      constexpr bool FIRST = decltype(first_step)::value;
      const uint8_t* const cur = lds + (s & 1) * STAGE;
      const uint8_t* const nxt = lds + ((s & 1) ^ 1) * STAGE;
      const uint32_t stage = base + (s & 1) * STAGE;
      // (between two pairs of matrix instructions at most two reads and a copy, which fit
      // their 64 cycles: a run of them would leave the matrix unit waiting)
#define FP8G_MFMA(I_, J_, H_)                                                                            \
  do {                                                                                                   \
    const v16i c_ = FIRST && H_ == 0 ? v16i{} : acc[I_][J_];                                             \
    acc[I_][J_] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bf[J_][H_].lo, af[I_][H_].lo, c_, 0, 0, 0);      \
    /* (a pure instruction: without this it is moved to where it is used) */                             \
    asm volatile("" : "+a"(acc[I_][J_]));                                                                \
    acc[I_][J_] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bf[J_][H_].hi, af[I_][H_].hi, acc[I_][J_], 0, 0, \
                                                        0);                                              \
    asm volatile("" : "+a"(acc[I_][J_]));                                                                \
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
      // second half: each fragment of a against 2 and 3 of b, after which the next step's
      // takes its place
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        const int i = m >> 2, h = (m >> 1) & 1, j = 2 + (m & 1);
        if (m < 4) bf[m >> 1][m & 1] = read_frag(nxt + ob, m >> 1, m & 1, lane);
        FP8G_MFMA(i, j, h);
        if (m % 2 == 1) issue(pl, a, tp, p_kb, stage, wave, EARLY_FIRST + m / 2);
        // (the half of this fragment that is done with)
        if (m % 2 == 1) af[i][h] = read_frag(nxt + oa, i, h, lane);
      }
#undef FP8G_MFMA
      advance();
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
    for (int k = 1; k < steps; ++k) step(std::false_type{});
    pin();
    const bool full = tc.mv == TS && tc.nv == TS;
    fresh = full ? 3 : 0;
    // A lane holds, of a's position pos, 16 positions of each fragment j of b: for every t 8
    // adjacent columns (u = 0) and, 16 further, 8 more (u = 1); the other half of the wave
    // holds the 8 after each. Exchanging u = 1 of lanes 0-15 (32-47) with u = 0 of lanes 16-31
    // (48-63) gives four lanes 64 bytes of a row, and exchanging t + 1 of lanes 0-7 of each 16
    // with t of lanes 8-15 gives eight lanes its 128: whole lines, non-temporal, eight rows a
    // store.
    const int l16 = lane & 15, q16 = lane >> 4;
    const int cl = wn * 128 + (l16 >> 3) * 32 + (q16 & 1) * 16 + (q16 >> 1) * 8;
    const int rl = wm * 128 + (l16 & 7) * 4;
    uint16_t* const d0 = tc.d + (int64_t)rl * a.N + cl;
    float sa[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sa[i] = tc.sa[min(wm * 128 + (lane & 31) * 4 + i, tc.mv - 1)];
#pragma unroll
    for (int t2 = 0; t2 < 2; ++t2) {
      float sb[2][2][8];                               // of the 8 columns of [t - 2 t2][u]
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // (columns come in eights, of which all or none exist)
          const int c0 = wn * 128 + (2 * t2 + tt) * 32 + u * 16 + (lane >> 5) * 8;
          const float* const from = tc.sb + min(c0, tc.nv - 8);
#pragma unroll
          for (int x = 0; x < 8; ++x) sb[tt][u][x] = from[x];
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t v[2][2][4];                           // [t - 2 t2][u]
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int q = 4 * (2 * t2 + tt) + 2 * u + (w >> 1), j = (w & 1) * 2;
              v[tt][u][w] = bf16_pair((float)acc[i][j][q] * sa[i] * sb[tt][u][2 * w],
                                      (float)acc[i][j + 1][q] * sa[i] * sb[tt][u][2 * w + 1]);
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
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // (no copy may arrive after the workgroup's LDS is someone else's)
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
}

// ---------------------------------------------------------------------------
// Smaller tiles, 64 FM x 64 FN by four waves of 32 FM x 32 FN, RING LDS stages, one tile a
// workgroup: a step's fragments are read during the one before, and its copies issued
// RING - 1/2 steps ahead. One barrier a step, half way: it publishes the stage that has landed
// and frees the one whose fragments are all in registers. Position r of fragment i of a wave's
// rows is row FM r + i (columns likewise), so that a lane's results are runs of 4 FN columns.
// Bound by a step's reads of LDS and its barrier: 0.7 of a 256x256 tile's rate, a loss smaller than that
// of CUs without work where 256x256 tiles are few (see kCost). 777x2064x1040 takes 11.3 us, of which 6
// are the launch and the pipeline's first and last steps.
template <int FM, int FN, int RING>
struct Ring {
  static constexpr int TM = 64 * FM, TN = 64 * FN, STAGE_BYTES = (TM + TN) * 128, BYTES = RING * STAGE_BYTES;
  static_assert(sizeof(Experts) <= BYTES, "the list of experts fits the stages' place");
};

// The tile of mv rows from `row` (of a, sa and d) and nv columns from n0 of expert g.
template <int FM, int FN, int RING, bool KTAIL>
__device__ __forceinline__ void ring_tile(const Int8Args& a, uint8_t* lds, int64_t g, int64_t row, int mv,
                                          int64_t n0, int nv) {
  constexpr int TM = 64 * FM;
  constexpr int RSTAGE = Ring<FM, FN, RING>::STAGE_BYTES;
  constexpr int PER = (TM + 64 * FN) / 32;             // a wave's copies of a stage, 8 rows each
  constexpr int PAIRS = FM * FN;                       // pairs of matrix instructions in half a step
  static_assert(PER % 2 == 0 && PER / 2 <= 2 * PAIRS, "copies between matrix instructions");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int steps = (int)((a.K + 127) / 128), kr = (int)(a.K % 128);
  // copy c: LDS rows 8 q .. +7 of the stage, q = wave PER + c, a's first
  const int8_t* const pa = a.a + row * a.K;
  const int8_t* const pb = a.b + (g * a.N + n0) * a.K;
  uint32_t voff[PER], past[2];
#pragma unroll
  for (int c = 0; c < PER; ++c) {
    const int q = wave * PER + c;
    const bool is_a = q < TM / 8;
    const int p = is_a ? q : q - TM / 8, F = is_a ? FM : FN;
    const int r = p / (4 * F) * (32 * F) + ((p & 3) * 8 + (lane >> 3)) * F + (p >> 2) % F;
    voff[c] = (uint32_t)min(r, (is_a ? mv : nv) - 1) * (uint32_t)a.K +
              (uint32_t)((lane & 7) ^ (lane >> 3) ^ (p & 1)) * 16u;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int chunk = ((lane & 7) ^ (lane >> 3) ^ q) * 16;
    past[q] = KTAIL && chunk >= kr ? (uint32_t)(chunk - (kr - 16)) : 0u;
  }
  const uint32_t base = lds_addr(lds);
  // (past the end the last step's again, for nothing: every wait counts alike; in a partial
  // last block a chunk past K is one that exists, which is masked later. PER is even, so copy
  // c's rows have the parity of c.)
  auto copy = [&](int s, int c) __attribute__((always_inline)) {
    const int kb = min(s, steps - 1), q = wave * PER + c;
    const uint32_t back = KTAIL && kb == steps - 1 ? past[c & 1] : 0u;
    copy16((q < TM / 8 ? pa : pb) + (int64_t)kb * 128, voff[c] - back,
           base + (uint32_t)(s % RING) * RSTAGE + (uint32_t)q * 1024u);
  };
  const int wm = (wave >> 1) * 32 * FM, wn = (wave & 1) * 32 * FN;
  int keep[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 2; ++q) keep[h][q] = (h * 4 + (lane >> 5) * 2 + q) * 16 < kr ? -1 : 0;
  const auto read_a = [&](const uint8_t* stage, int i, int h, bool last_block) __attribute__((always_inline)) {
    Frag f = read_frag(stage + wm * 128, i, h, lane);
    if constexpr (KTAIL) {
      f.lo &= last_block ? keep[h][0] : -1;
      f.hi &= last_block ? keep[h][1] : -1;
    }
    return f;
  };
  const auto read_b = [&](const uint8_t* stage, int j, int h) __attribute__((always_inline)) {
    return read_frag(stage + (TM + wn) * 128, j, h, lane);
  };
  // own reads and copies of long enough ago have arrived; then everyone's have
  auto meet = [&](auto n) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_waitcnt(vmcnt_only(decltype(n)::value));
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  v16i acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = v16i{};
#pragma unroll
  for (int c = 0; c < (RING - 1) * PER + PER / 2; ++c) copy(c / PER, c % PER);
  meet(std::integral_constant<int, (RING - 2) * PER + PER / 2>{});
  Frag fa[FM][2], fb[FN][2];                           // [fragment][half of the 128 bytes]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i][h] = read_a(lds, i, h, steps == 1);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j][h] = read_b(lds, j, h);
  }
  for (int s = 0; s < steps; ++s) {
    const bool last_next = s + 1 == steps - 1;
    // (the empty asm keeps a pure instruction from moving to where it is used)
#define FP8G_MFMA(I_, J_, A_, B_)                                                               \
  do {                                                                                          \
    acc[I_][J_] = __builtin_amdgcn_mfma_i32_32x32x32_i8(B_.lo, A_.lo, acc[I_][J_], 0, 0, 0);    \
    asm volatile("" : "+a"(acc[I_][J_]));                                                       \
    acc[I_][J_] = __builtin_amdgcn_mfma_i32_32x32x32_i8(B_.hi, A_.hi, acc[I_][J_], 0, 0, 0);    \
    asm volatile("" : "+a"(acc[I_][J_]));                                                       \
  } while (0)
#pragma unroll
    for (int m = 0; m < PAIRS; ++m) {
      const int i = m / FN, j = m % FN;
      FP8G_MFMA(i, j, fa[i][0], fb[j][0]);
#pragma unroll
      for (int c = m * (PER / 2) / PAIRS; c < (m + 1) * (PER / 2) / PAIRS; ++c) copy(s + RING - 1, PER / 2 + c);
    }
    // this stage has been read by all, and the next one's copies have landed: those of
    // RING - 2 steps may be on their way
    meet(std::integral_constant<int, (RING - 2) * PER>{});
    const uint8_t* const st = lds + ((s + 1) % RING) * RSTAGE;
#pragma unroll
    for (int m = 0; m < PAIRS; ++m) {
      const int i = m / FN, j = m % FN;
      // (the first halves are done with)
#pragma unroll
      for (int r = m * (FM + FN) / PAIRS; r < (m + 1) * (FM + FN) / PAIRS; ++r) {
        if (r < FM) fa[r][0] = read_a(st, r, 0, last_next);
        else fb[r - FM][0] = read_b(st, r - FM, 0);
      }
      FP8G_MFMA(i, j, fa[i][1], fb[j][1]);
#pragma unroll
      for (int c = m * (PER / 2) / PAIRS; c < (m + 1) * (PER / 2) / PAIRS; ++c) copy(s + RING, c);
    }
#undef FP8G_MFMA
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i][1] = read_a(st, i, 1, last_next);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[j][1] = read_b(st, j, 1);
  }
  // (no copy may arrive after the workgroup's LDS is someone else's)
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
  // b is the first operand: lane l holds position l % 32 of fragment i of a, and of fragment j
  // of b positions 8 t + 4 (l / 32) + e; column FN position + j
  uint16_t* const d = a.d + row * a.N + n0;
  const float* const psb = a.sb + g * a.N + n0;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
#pragma unroll
    for (int h = 0; h < FN / 2; ++h) {                 // 8 columns at a time: 8 / FN positions
      const int col = wn + t * 8 * FN + (lane >> 5) * 4 * FN + h * 8;
      if (col >= nv) continue;
      float sb[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) sb[x] = psb[col + x];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int r = wm + (lane & 31) * FM + i;
        if (r >= mv) continue;
        const float sa = a.sa[row + r];
        u32x4 v;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int x = h * 8 + 2 * w, e = x / FN, j = x % FN;
          v[w] = bf16_pair((float)acc[i][j][4 * t + e] * sa * sb[2 * w],
                           (float)acc[i][j + 1][4 * t + e] * sa * sb[2 * w + 1]);
        }
        *reinterpret_cast<u32x4*>(d + (int64_t)r * a.N + col) = v;
      }
    }
  }
}

// Workgroups are dealt to the 8 XCDs in turn: an XCD's get a run of tiles.
__device__ __forceinline__ int xcd_run(int w, int tiles) {
  const int x = w & 7, most = tiles >> 3, more = tiles & 7;
  return x * most + min(x, more) + (w >> 3);
}

// Tile `at` of a launch's (rows of `side`): its expert, the expert's first row and rows, the tile's place.
struct Place {
  int64_t g, row;
  int rows, mb, nb;
};
__device__ __forceinline__ int list_tiles(const Int8Args& a, Experts& ex, int side, int nblocks) {
  if (a.mode == MODE_DENSE) return (int)((a.rows + side - 1) / side) * nblocks;
  if (threadIdx.x < 64) list_experts(a, ex, side, threadIdx.x);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(ex.before[ex.n]) * nblocks;
}
__device__ __forceinline__ Place place_of(const Int8Args& a, const Experts& ex, int at, int side, int nblocks, int swizzle) {
  Place p = {0, 0, (int)a.rows, 0, 0};
  int before = 0, mblocks = (int)((a.rows + side - 1) / side);
  if (a.mode != MODE_DENSE) {
    int lo = 0, hi = __builtin_amdgcn_readfirstlane(ex.n) - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (at / nblocks < __builtin_amdgcn_readfirstlane(ex.before[mid + 1])) hi = mid;
      else lo = mid + 1;
    }
    before = __builtin_amdgcn_readfirstlane(ex.before[lo]);
    mblocks = __builtin_amdgcn_readfirstlane(ex.before[lo + 1]) - before;
    p.g = __builtin_amdgcn_readfirstlane(ex.id[lo]);
    p.rows = __builtin_amdgcn_readfirstlane(ex.rows[lo]);
    p.row = a.mode == MODE_MASKED ? p.g * a.rows : __builtin_amdgcn_readfirstlane(ex.row0[lo]);
    __syncthreads();                                   // (read by all: the copies may come)
  }
  gidx::swizzle_tile(at - before * nblocks, mblocks, nblocks, swizzle, p.mb, p.nb);
  return p;
}

template <int FM, int FN, int RING, bool KTAIL>
__global__ void __launch_bounds__(256, 1)
int8_ring_kernel(Int8Args a, int nblocks) {
  using R = Ring<FM, FN, RING>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[R::BYTES];
  Experts& ex = *reinterpret_cast<Experts*>(lds);
  const int tiles = list_tiles(a, ex, R::TM, nblocks);
  if ((int)blockIdx.x >= tiles) return;
  const Place p = place_of(a, ex, xcd_run(blockIdx.x, tiles), R::TM, nblocks, 8);
  const int64_t m0 = (int64_t)p.mb * R::TM, n0 = (int64_t)p.nb * R::TN;
  ring_tile<FM, FN, RING, KTAIL>(a, lds, p.g, p.row + m0, (int)min((int64_t)R::TM, p.rows - m0), n0,
                                 (int)min((int64_t)R::TN, a.N - n0));
}

// The tiles that int8_tile_kernel leaves, in quarters where these are no more than the CUs, else in
// halves of 128 columns.
__global__ void __launch_bounds__(256, 1)
int8_rest_kernel(Int8Args a, int nblocks) {
  using Half = Ring<4, 2, 3>;
  using Quarter = Ring<2, 2, 4>;
  static_assert(Half::TM == TS && 2 * Half::TN == TS && 2 * Quarter::TM == TS && 2 * Quarter::TN == TS, "parts of the tiles");
  __shared__ __attribute__((aligned(16))) uint8_t lds[Half::BYTES > Quarter::BYTES ? Half::BYTES : Quarter::BYTES];
  Experts& ex = *reinterpret_cast<Experts*>(lds);
  const int tiles = list_tiles(a, ex, TS, nblocks);
  const int done = (int)full_rounds(tiles, a.round), rest = tiles - done;
  const int cut = 4 * rest <= a.round ? 4 : 2;
  if ((int)blockIdx.x >= cut * rest) return;
  const int h = xcd_run(blockIdx.x, cut * rest);
  const Place p = place_of(a, ex, done + h / cut, TS, nblocks, 4);
  const int64_t m0 = (int64_t)p.mb * TS + (cut == 4 ? h % 4 / 2 * Quarter::TM : 0), n0 = (int64_t)p.nb * TS + h % 2 * Half::TN;
  if (m0 >= p.rows || n0 >= a.N) return;               // (uniform over the workgroup)
  const int nv = (int)min((int64_t)Half::TN, a.N - n0);
  if (cut == 4) ring_tile<2, 2, 4, false>(a, lds, p.g, p.row + m0, (int)min((int64_t)Quarter::TM, p.rows - m0), n0, nv);
  else ring_tile<4, 2, 3, false>(a, lds, p.g, p.row + m0, (int)min((int64_t)TS, p.rows - m0), n0, nv);
}

// ---------------------------------------------------------------------------
// Few rows: the work is streaming b, and a again for every column block. A workgroup owns
// 16 NT output columns and up to 16 MT rows; its four waves take the 128-byte blocks of K in
// turn, each with a ring of DEPTH stages of its own in LDS, so that no wave waits for another
// until their sums meet; two or three workgroups on a CU rather than a deeper ring, which overlaps
// their starts and ends too (16x28672x4096 26.3 us with 3 stages, 37.4 with 8; 32x14336x4096 15.9 with 2,
// 18.7 with 5; 512x4096x4096 16.8 with one, 19.8 with 2). Whole 128-byte lines go straight into LDS:
// the same fragments loaded from global memory into registers touch 16 lines of which they take half,
// and cost twice the cycles. Bound by HBM and by the latency of the first and last steps: 16x4096x7168
// 8.0 us, 16x8192x8192 15.1, 4.4 TB/s (128x128 tiles 26 and 30).
constexpr int SK_WAVES = 4;

template <int MT, int NT, int DEPTH, bool KTAIL>
__global__ void __launch_bounds__(SK_WAVES * 64, 1)
int8_skinny_kernel(Int8Args a) {
  constexpr int PIECE = 16 * 128;                      // 16 rows of a stage
  constexpr int SK_STAGE = (MT + NT) * PIECE, PER = 2 * (MT + NT);
  static_assert(SK_WAVES * MT * NT * 1024 <= SK_WAVES * DEPTH * SK_STAGE, "the sums fit the ring");
  __shared__ __attribute__((aligned(16))) uint8_t lds[SK_WAVES * DEPTH * SK_STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nblocks = (int)((a.N + 16 * NT - 1) / (16 * NT));
  const int64_t n0 = (int64_t)((int)blockIdx.x % nblocks) * (16 * NT), m0 = (int64_t)((int)blockIdx.x / nblocks) * (16 * MT);
  const int mv = (int)min((int64_t)16 * MT, a.rows - m0), nv = (int)min((int64_t)16 * NT, a.N - n0);
  const int nkb = (int)((a.K + 127) / 128), kr = (int)(a.K % 128);
  const int8_t* const pa = a.a + m0 * a.K;
  const int8_t* const pb = a.b + n0 * a.K;
  // copy c: 8 rows of the stage's 16 (MT + NT), a's first; rows past the last are copies of it
  uint32_t voff[PER], past[2];
#pragma unroll
  for (int c = 0; c < PER; ++c) {
    const int r = (c < 2 * MT ? c : c - 2 * MT) * 8 + (lane >> 3);
    voff[c] = (uint32_t)min(r, (c < 2 * MT ? mv : nv) - 1) * (uint32_t)a.K +
              (uint32_t)((lane & 7) ^ (lane >> 3) ^ (c & 1)) * 16u;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int chunk = ((lane & 7) ^ (lane >> 3) ^ q) * 16;
    past[q] = KTAIL && chunk >= kr ? (uint32_t)(chunk - (kr - 16)) : 0u;
  }
  const uint32_t base = lds_addr(lds) + (uint32_t)wave * (DEPTH * SK_STAGE);
  const uint8_t* const ring = lds + wave * (DEPTH * SK_STAGE);
  // (past the end the last block again, for nothing: every wait counts alike; in a partial last
  // block a chunk past K is one that exists, which is masked later)
  const auto copy = [&](int s, int slot) __attribute__((always_inline)) {
    const int kb = min(wave + s * SK_WAVES, nkb - 1);
    const bool tail = KTAIL && kb == nkb - 1;
#pragma unroll
    for (int c = 0; c < PER; ++c)
      copy16((c < 2 * MT ? pa : pb) + (int64_t)kb * 128, voff[c] - (tail ? past[c & 1] : 0u),
             base + (uint32_t)(slot * SK_STAGE + c * 1024));
  };
  const auto frag = [&](const uint8_t* piece) __attribute__((always_inline)) {
    const int r = lane & 15, c = (lane >> 4) * 2;
    Frag v;
    v.lo = *reinterpret_cast<const v4i*>(piece + r * 128 + swz(r, c) * 16);
    v.hi = *reinterpret_cast<const v4i*>(piece + r * 128 + swz(r, c + 1) * 16);
    return v;
  };
  const int keep[2] = {(lane >> 4) * 32 < kr ? -1 : 0, (lane >> 4) * 32 + 16 < kr ? -1 : 0};
  v4i acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  const int steps = nkb > wave ? (nkb - wave + SK_WAVES - 1) / SK_WAVES : 0;
#pragma unroll
  for (int s = 0; s < DEPTH; ++s) copy(s, s);
  int slot = 0;
  for (int s = 0; s < steps; ++s) {
    __builtin_amdgcn_s_waitcnt(vmcnt_only((DEPTH - 1) * PER));
    asm volatile("" ::: "memory");
    const uint8_t* const st = ring + slot * SK_STAGE;
    Frag fa[MT], fb[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) fb[j] = frag(st + (MT + j) * PIECE);
#pragma unroll
    for (int i = 0; i < MT; ++i) fa[i] = frag(st + i * PIECE);
    if constexpr (KTAIL) {
      const bool tail = wave + s * SK_WAVES == nkb - 1;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        fb[j].lo &= tail ? keep[0] : -1;
        fb[j].hi &= tail ? keep[1] : -1;
      }
    }
    // this stage is in registers: the copies of the one DEPTH on take its place
    __builtin_amdgcn_s_waitcnt(0xC07F);                // lgkmcnt(0)
    __builtin_amdgcn_sched_barrier(0);
    copy(s + DEPTH, slot);
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j].lo, fa[i].lo, acc[i][j], 0, 0, 0);
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j].hi, fa[i].hi, acc[i][j], 0, 0, 0);
      }
  }
  // (no copy may arrive any more: the sums take the ring's place)
  __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
  __syncthreads();
  v4i* const red = reinterpret_cast<v4i*>(lds);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[(wave * MT * NT + i * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // (b is the first operand: lane l holds row l % 16 and columns 4 (l / 16) .. +3)
  for (int t = wave; t < MT * NT; t += SK_WAVES) {
    v4i sum = red[t * 64 + lane];
#pragma unroll
    for (int v = 1; v < SK_WAVES; ++v) sum += red[(v * MT * NT + t) * 64 + lane];
    const int r = (t / NT) * 16 + (lane & 15), c = (t % NT) * 16 + (lane >> 4) * 4;
    if (r >= mv || c >= nv) continue;
    const float sa = a.sa[m0 + r];
    const float* const sb = a.sb + n0 + c;
    Pack<uint32_t, 2> o;
    o.v[0] = bf16_pair((float)sum[0] * sa * sb[0], (float)sum[1] * sa * sb[1]);
    o.v[1] = bf16_pair((float)sum[2] * sa * sb[2], (float)sum[3] * sa * sb[3]);
    *reinterpret_cast<Pack<uint32_t, 2>*>(a.d + (m0 + r) * a.N + n0 + c) = o;
  }
}

// The kernels, from few rows to many. A launch takes `start`, for each 128 bytes of K `deep`, and for each
// round of workgroups over the CUs `round` and for each 128 bytes of K `block`, or `odd` where K is not a
// multiple of 128 (rows then start inside a 128-byte line, and a copy touches two lines for one), in ns. Of
// the first three kernels several workgroups fit a CU: their rounds are a quotient, those of the others
// whole numbers. A TILE256 launch's short last round is in RING128's or RING256's parts. Fitted to 400
// products of M 1 to 3000 and 200 of 8 to 9000, N 256 to 28,800, K 256 to 8960, weights cold (each kernel
// within 8 to 13% rms). The smallest estimate picks within 1.2% of the fastest on the geometric mean and
// within 28% at most (126x448x2304, 4.9 us).
enum Kernel { SKINNY16, SKINNY32, SKINNY64, RING128, RING256, TILE256, KERNELS };
struct Cost {
  int tm, tn;
  int64_t start, deep, round, block, odd;
};
constexpr Cost kCost[KERNELS] = {
    {16, 16, 2700, 20, 460, 67, 68},  {32, 32, 2900, 46, 780, 129, 157}, {64, 64, 3600, 130, 1210, 263, 340},
    {128, 128, 300, 0, 5500, 380, 510}, {256, 128, 0, 0, 8900, 650, 830}, {256, 256, 0, 0, 10000, 1120, 0},
};

int64_t blocks(int64_t n, int64_t side) { return (n + side - 1) / side; }

// Row blocks of a launch over all experts, or a bound on them.
int64_t row_blocks(const Int8Args& a, int side) {
  const int64_t mb = blocks(a.rows, side);
  return a.mode == MODE_DENSE ? mb : (a.mode == MODE_MASKED ? mb * a.G : mb + a.G);
}

Kernel choose(const Int8Args& a, int expected_m, int cus) {
  if (a.mode != MODE_DENSE) {
    // 128-row blocks where an expert's rows are likely to be one of them, or where they do not
    // fill the CUs once (8 experts 4096x7168 of 64 tokens each 40 / 70 us with 256-row blocks, 32
    // slabs of 32 rows 7168x2048 108 / 130; but 32 experts 4096x2048 of 128 tokens on average, of
    // which half take two blocks, 104 / 69).
    const bool one = a.mode == MODE_CONTIGUOUS ? a.rows <= (int64_t)128 * a.G
                                               : (expected_m > 0 ? expected_m <= 96 : a.rows <= 128);
    if (one || row_blocks(a, 128) * blocks(a.N, 128) <= cus) return RING128;
    return a.K % 128 ? RING256 : TILE256;
  }
  int best = RING128;
  int64_t least = INT64_MAX;
  for (int k = 0; k < (a.K % 128 ? TILE256 : KERNELS); ++k) {
    const Cost& c = kCost[k];
    const int64_t tiles = blocks(a.rows, c.tm) * blocks(a.N, c.tn);
    if (tiles >= (1 << 24)) continue;                  // (2^32 threads; 128x128 tiles are fewer: checked before)
    const int64_t kb = blocks(a.K, 128), last = k == TILE256 ? tiles - full_rounds(tiles, cus) : 0;
    const int64_t round = c.round + (a.K % 128 ? c.odd : c.block) * kb;
    int64_t t = c.start + c.deep * kb + (k <= SKINNY64 ? tiles * round / cus : blocks(tiles - last, cus) * round);
    const Cost& r = kCost[4 * last <= cus ? RING128 : RING256];
    if (last) t += r.start + r.round + r.block * kb;
    if (t < least) {
      least = t;
      best = k;
    }
  }
  return (Kernel)best;
}

typedef void (*SkinnyFn)(Int8Args);
typedef void (*TilesFn)(Int8Args, int);
SkinnyFn skinny_pick(Kernel k, bool tail) {
  if (k == SKINNY16) return tail ? int8_skinny_kernel<1, 1, 3, true> : int8_skinny_kernel<1, 1, 3, false>;
  if (k == SKINNY32) return tail ? int8_skinny_kernel<2, 2, 2, true> : int8_skinny_kernel<2, 2, 2, false>;
  return tail ? int8_skinny_kernel<4, 4, 1, true> : int8_skinny_kernel<4, 4, 1, false>;
}
TilesFn ring_pick(Kernel k, bool tail) {
  if (k == RING128) return tail ? int8_ring_kernel<2, 2, 4, true> : int8_ring_kernel<2, 2, 4, false>;
  return tail ? int8_ring_kernel<4, 2, 3, true> : int8_ring_kernel<4, 2, 3, false>;
}

}  // namespace

hipError_t launch_int8_quantize(const void* x, int type, int64_t rows, int64_t cols, int64_t ldx, int8_t* q,
                                int64_t ldq, float* scales, hipStream_t stream) {
  if (type == TYPE_F32) return quant_launch<float>(x, rows, cols, ldx, q, ldq, scales, stream);
  if (type == TYPE_BF16) return quant_launch<bf16_t>(x, rows, cols, ldx, q, ldq, scales, stream);
  return quant_launch<f16_t>(x, rows, cols, ldx, q, ldq, scales, stream);
}

hipError_t launch_int8(const Int8Args& args, const DeviceInfo& dev, int expected_m, hipStream_t stream) {
  const Kernel k = choose(args, expected_m, dev.cu_count);
  const bool tail = args.K % 128 != 0;
  const int64_t nb = blocks(args.N, kCost[k].tn), tiles = row_blocks(args, kCost[k].tm) * nb;
  if (k <= SKINNY64) {
    skinny_pick(k, tail)<<<dim3((unsigned)tiles), dim3(64 * SK_WAVES), 0, stream>>>(args);
  } else if (k != TILE256) {
    ring_pick(k, tail)<<<dim3((unsigned)tiles), dim3(256), 0, stream>>>(args, (int)nb);
  } else {
    Int8Args all = args;
    all.round = dev.cu_count;
    // (grouped: how many tiles there are is known on the device alone; a launch for what may be left)
    if (args.mode != MODE_DENSE || full_rounds(tiles, all.round) > 0) {
      const int64_t grid = tiles < dev.cu_count ? tiles : dev.cu_count;
      int8_tile_kernel<<<dim3((unsigned)grid), dim3(256), 0, stream>>>(all, (int)nb, grid % 8 == 0 ? 1 : 0);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    // (at most round / 2 tiles: their parts are no more than a round)
    const int64_t rest = args.mode != MODE_DENSE ? tiles : tiles - full_rounds(tiles, all.round);
    const int64_t parts = 4 * rest < all.round ? 4 * rest : all.round;
    if (rest > 0) int8_rest_kernel<<<dim3((unsigned)parts), dim3(256), 0, stream>>>(all, (int)nb);
  }
  return hipGetLastError();
}

void int8_kernels(std::vector<const void*>& out) {
  int per;
  for (int64_t cols : {16, 1024, 2048, 8192, 16384, 32768}) {
    out.push_back((const void*)quant_pick<float>(cols, &per));
    out.push_back((const void*)quant_pick<bf16_t>(cols, &per));
    out.push_back((const void*)quant_pick<f16_t>(cols, &per));
  }
  for (bool tail : {false, true}) {
    for (Kernel k : {SKINNY16, SKINNY32, SKINNY64}) out.push_back((const void*)skinny_pick(k, tail));
    for (Kernel k : {RING128, RING256}) out.push_back((const void*)ring_pick(k, tail));
  }
  out.push_back((const void*)int8_tile_kernel);
  out.push_back((const void*)int8_rest_kernel);
}

}  // namespace fp8g
