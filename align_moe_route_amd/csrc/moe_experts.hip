// Products grouped by expert in 16 bits, forward and backward, over the route-sort
// metadata, MI355X (gfx950, CDNA4, wave64).  Definitions: include/moe_experts.h.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "half.h"
#include "moe_experts.h"
#include "moe_route_sort.h"

namespace {

// The three directions are one tiled product C[i, j] = sum_c A[i, c] B[j, c]:
//   kForward  i sorted rows, j = n, c = k: A = x (rows along c), B = w (rows along c)
//   kRows     i sorted rows, j = k, c = n: A = dy (rows along c), B = w (rows along j)
//   kWeights  i = n, j = k, c sorted rows of one expert: A = dy (rows along i), B = x
//             (rows along j)
enum Dir { kForward, kRows, kWeights };

struct GArgs {
  const uint16_t *a, *b;
  const int32_t *sid, *eob, *npp;
  void* out;
  int routes, k, E, block, sorted;
  int I, J, C;    // sizes of i, j, c (I: kWeights only; C: the others only)
  int row_limit;  // rows the metadata can hold: (max_rows / block) * block
  int nrt, nct;   // tiles of i (over all sorted rows, or of one expert), tiles of j
  int run;        // consecutive row tiles of an XCD
};

constexpr int kThreads = 256, kWaves = 4;
constexpr int kStep = 64;  // of c

// Operand tiles in LDS, in 16-byte chunks of eight values.
//
// Rows along c: 8 chunks a row, the chunk at slot p of row r is p ^ (r & 7) ^ (r >> 3 &
// 1), so that the 32 rows of an operand read hit distinct banks.
//
// Rows along the tile (one LDS row per c, W values wide): read by ds_read_b64_tr_b16,
// in which 16 lanes together read four rows of 16 values and each lane receives one
// column's four values.  Slot p of row c holds chunk p ^ (c & 3) << 2: the four rows
// that 32 lanes read 64 bytes of lie on distinct banks.
__device__ __forceinline__ int swz(int r, int p) { return p ^ (r & 7) ^ ((r >> 3) & 1); }
template <int W>
__device__ __forceinline__ int swz_across(int c, int p) {
  static_assert(W >= 128, "chunk moves within the row");
  return p ^ ((c & 3) << 2);
}

typedef __attribute__((address_space(3))) char* lds_t;
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x2 read_turned(const char* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4*)(lds_t) const_cast<char*>(p)));
}

// Operand of v_mfma_*_32x32x16: lane l holds values 8 (l / 32) .. + 7 of c of row l mod
// 32; rows m0 .., c from 16 kk.
template <bool ACROSS, int W>
__device__ __forceinline__ u32x4 operand(const u32x4* tile, int m0, int kk) {
  const int lane = threadIdx.x & 63;
  if constexpr (!ACROSS) {
    const int r = m0 + (lane & 31);
    return tile[r * 8 + swz(r, kk * 2 + (lane >> 5))];
  } else {
    const int c = kk * 16 + (lane >> 5) * 8 + ((lane & 15) >> 2);
    const int m = m0 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
    const char* p = reinterpret_cast<const char*>(tile + c * (W / 8) + swz_across<W>(c, m / 8)) + (m & 4) * 2;
    const u32x2 lo = read_turned(p), hi = read_turned(p + 4 * (W / 8) * 16);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  }
}

// First block of [0, n) whose expert is at least e (found for e and e + 1), by 64-ary
// search: the experts of used blocks ascend.
__device__ __forceinline__ void segment(const int32_t* eob, int n, int e, int& first, int& last) {
  const int lane = threadIdx.x & 63;
  auto lower = [&](int key) {
    int lo = 0, len = n;  // the answer lies in [lo, lo + len]
    while (len > 0) {
      const int step = (len + 63) / 64, at = lo + lane * step;
      const bool less = lane * step < len && eob[at] < key;
      const int c = __builtin_popcountll(__ballot(less));  // probes 0 .. c - 1 are less
      if (c == 0) return lo;
      const int from = (c - 1) * step + 1;
      lo += from;
      len = min(step - 1, len - from);
    }
    return lo;
  };
  first = lower(e);
  last = lower(e + 1);
}

constexpr int kXcds = 8;

template <int BM>
constexpr int tile_rows() {
  return BM < 32 ? 32 : BM;
}

template <int DIR, int BM, int BN>
struct Tile {
  static constexpr int kRows = tile_rows<BM>();
  u32x4 a[kRows * kStep / 8], b[BN * kStep / 8];
  int32_t row[DIR == kWeights ? kStep * 2 : kRows];
};

template <typename H, int DIR, int BM, int BN, bool F32>
__global__ __launch_bounds__(kThreads, 2) void k_product(GArgs g) {
  constexpr bool kAcrossA = DIR == kWeights, kAcrossB = DIR != kForward;
  constexpr int TR = tile_rows<BM>();
  constexpr int WI = BM >= 128 ? 2 : 1, WJ = kWaves / WI;  // waves along i and j
  constexpr int FM = TR / WI / 32, FN = BN / WJ / 32;
  constexpr int AP = TR * kStep / 8 / kThreads, BP = BN * kStep / 8 / kThreads;  // chunks a thread stages in a step
  __shared__ Tile<DIR, BM, BN> l;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int npp = min(*g.npp, g.row_limit);

  int i0, j0, e, c_first = 0, c_end;  // the tile, its expert, the range of c
  uint64_t has[2] = {~0ull, ~0ull};   // rows that hold a slot
  if constexpr (DIR == kWeights) {
    const int h = blockIdx.x, x = h % kXcds, j = h / kXcds, each = g.nrt * g.nct;
    e = j / each * kXcds + x;
    if (e >= g.E) return;
    i0 = j % each / g.nct * BM, j0 = j % each % g.nct * BN;
    int first, last;
    segment(g.eob, max(npp, 0) / g.block, e, first, last);
    c_first = first * g.block, c_end = last * g.block;
  } else {
    const int h = blockIdx.x, x = h % kXcds, j = h / kXcds, i = j / g.nct;
    const int rt = (i / g.run * kXcds + x) * g.run + i % g.run;
    if (rt >= g.nrt) return;
    i0 = rt * BM, j0 = j % g.nct * BN;
    if (i0 + BM > npp) return;  // npp is a multiple of block and BM divides block
    e = g.eob[i0 / g.block];
    if (e < 0 || e >= g.E) return;
    c_end = g.C;
    if (tid < TR) {
      const int s = tid < BM ? g.sid[i0 + tid] : -1;
      const bool ok = s >= 0 && s < g.routes;
      l.row[tid] = !ok ? -1 : (DIR == kForward && !g.sorted) ? s / g.k : i0 + tid;
    }
    __syncthreads();
    has[0] = __ballot(lane < TR && l.row[lane % TR] >= 0);
    has[1] = TR > 64 ? __ballot(l.row[(64 + lane) % TR] >= 0) : 0;
  }
  e = __builtin_amdgcn_readfirstlane(e);

  const int64_t across = DIR == kRows ? (int64_t)e * g.C * g.J : 0;
  u32x4 ra[AP], rb[BP];
  // chunks of c from c0 into registers; whatever lies past an edge is zero
  auto load = [&](int c0) {
    if constexpr (!kAcrossA) {
      const int r = tid / 8, c = c0 + swz(r, tid % 8) * 8;  // swz: the same for rows r + 32 p
#pragma unroll
      for (int p = 0; p < AP; ++p) {
        const int row = l.row[r + p * 32];
        ra[p] = load8(g.a + (int64_t)row * g.C + c, row < 0 ? 0 : c_end - c);
      }
    } else {
      constexpr int W = BM / 8, S = kThreads / W;
#pragma unroll
      for (int p = 0; p < AP; ++p) {
        const int c = tid / W + p * S, i = i0 + swz_across<BM>(c, tid % W) * 8;
        const int r = c0 + c;
        const int s = r < c_end ? g.sid[r] : -1;
        ra[p] = load8(g.a + (int64_t)r * g.I + i, s < 0 || s >= g.routes ? 0 : g.I - i);
      }
    }
    if constexpr (!kAcrossB) {
      const int r = tid / 8, c = c0 + swz(r, tid % 8) * 8;
#pragma unroll
      for (int p = 0; p < BP; ++p) {
        const int j = j0 + r + p * 32;
        rb[p] = load8(g.b + ((int64_t)e * g.J + j) * g.C + c, j < g.J ? c_end - c : 0);
      }
    } else {
      constexpr int W = BN / 8, S = kThreads / W;
#pragma unroll
      for (int p = 0; p < BP; ++p) {
        const int c = tid / W + p * S, j = j0 + swz_across<BN>(c, tid % W) * 8;
        if constexpr (DIR == kRows) {
          rb[p] = load8(g.b + across + (int64_t)(c0 + c) * g.J + j, c0 + c < c_end ? g.J - j : 0);
        } else {
          const int r = c0 + c;
          const int s = r < c_end ? g.sid[r] : -1;
          const bool ok = s >= 0 && s < g.routes;
          const int64_t row = g.sorted ? r : ok ? s / g.k : 0;
          rb[p] = load8(g.b + row * g.J + j, ok ? g.J - j : 0);
        }
      }
    }
  };
  auto store = [&] {
#pragma unroll
    for (int p = 0; p < AP; ++p) l.a[tid + p * kThreads] = ra[p];
#pragma unroll
    for (int p = 0; p < BP; ++p) l.b[tid + p * kThreads] = rb[p];
  };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
  const int wi = wv / WJ * FM * 32, wj = wv % WJ * FN * 32;
  if (c_first < c_end) load(c_first);
  for (int c0 = c_first; c0 < c_end; c0 += kStep) {
    store();
    __syncthreads();
    if (c0 + kStep < c_end) load(c0 + kStep);
#pragma unroll
    for (int kk = 0; kk < kStep / 16; ++kk) {
      u32x4 fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[i] = operand<kAcrossA, TR>(l.a, wi + i * 32, kk);
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[j] = operand<kAcrossB, BN>(l.b, wj + j * 32, kk);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = H::mfma32(fb[j], fa[i], acc[i][j]);
    }
    __syncthreads();
  }

  // Result register v of lane l: column (of j) 8 (v / 4) + 4 (l / 32) + v mod 4, row (of i)
  // l mod 32.
  const int64_t base = DIR == kWeights ? (int64_t)e * g.I : 0;
  const int rows = DIR == kWeights ? g.I - i0 : BM;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = wi + i * 32 + (lane & 31);
    const bool ok = m >= 64 ? has[1] >> (m - 64) & 1 : has[0] >> m & 1;
    if (m >= rows) continue;
    const int64_t at = (base + i0 + m) * g.J;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; v += 2) {
        const int n = j0 + wj + j * 32 + 8 * (v / 4) + 4 * (lane >> 5) + v % 4;
        const float p = ok ? acc[i][j][v] : 0.0f, q = ok ? acc[i][j][v + 1] : 0.0f;
        if constexpr (F32) {
          float* o = static_cast<float*>(g.out) + at + n;
          if (n < g.J) o[0] = p;
          if (n + 1 < g.J) o[1] = q;
        } else {
          uint16_t* o = static_cast<uint16_t*>(g.out) + at + n;
          const uint32_t b = H::pack(p, q);
          if (n < g.J) o[0] = (uint16_t)b;
          if (n + 1 < g.J) o[1] = (uint16_t)(b >> 16);
        }
      }
  }
}

constexpr int kCols = 256;

template <typename H, int DIR, bool F32>
const void* product_kernel(int bm) {
  if constexpr (DIR == kWeights) {
    return reinterpret_cast<const void*>(k_product<H, DIR, 128, kCols, F32>);
  } else {
    switch (bm) {
      case 128: return reinterpret_cast<const void*>(k_product<H, DIR, 128, kCols, F32>);
      case 64: return reinterpret_cast<const void*>(k_product<H, DIR, 64, kCols, F32>);
      case 32: return reinterpret_cast<const void*>(k_product<H, DIR, 32, kCols, F32>);
      default: return reinterpret_cast<const void*>(k_product<H, DIR, 16, kCols, F32>);
    }
  }
}

template <int DIR>
const void* product_kernel(int dtype, bool f32, int bm) {
  if (dtype == MRS_DTYPE_BF16) return f32 ? product_kernel<BF16, DIR, true>(bm) : product_kernel<BF16, DIR, false>(bm);
  return f32 ? product_kernel<FP16, DIR, true>(bm) : product_kernel<FP16, DIR, false>(bm);
}

constexpr int kMaxCols = 1 << 20;

template <int DIR>
int product(const void* a, const void* b, int dtype, const int32_t* sid, const int32_t* eob, const int32_t* npp, int M,
            int k, int E, int K, int N, int block, int x_rows, int out_dtype, void* out, void* stream) {
  if (M < 0 || k < 1 || k > 64 || E < 1 || E > 4096 || K < 1 || K > kMaxCols || N < 1 || N > kMaxCols || block < 16 ||
      block % 16 != 0 || (dtype != MRS_DTYPE_BF16 && dtype != MRS_DTYPE_F16) ||
      (out_dtype != dtype && out_dtype != MRS_DTYPE_F32) || (x_rows != MRS_X_TOKENS && x_rows != MRS_X_SORTED))
    return MRS_ERR_INVALID_ARG;
  const int64_t max_rows = moe_route_sort_max_rows(M, E, k, block);
  if (max_rows < 0) return MRS_ERR_OVERFLOW;
  const int64_t row_limit = max_rows / block * block;
  if (row_limit == 0 && DIR != kWeights) return MRS_OK;  // no token: nothing to write
  if (!out || !npp || (row_limit > 0 && (!a || !b || !sid || !eob))) return MRS_ERR_NULL_POINTER;
  if (!aligned_to(a, 2) || !aligned_to(b, 2) || !aligned_to(out, out_dtype == MRS_DTYPE_F32 ? 4 : 2) ||
      !aligned_to(sid, 4) || !aligned_to(eob, 4) || !aligned_to(npp, 4))
    return MRS_ERR_MISALIGNED;
  GArgs g{};
  g.a = static_cast<const uint16_t*>(a), g.b = static_cast<const uint16_t*>(b);
  g.sid = sid, g.eob = eob, g.npp = npp, g.out = out;
  g.routes = M * k, g.k = k, g.E = E, g.block = block, g.sorted = x_rows == MRS_X_SORTED;
  g.row_limit = (int)row_limit;
  int bm;
  int64_t grid;
  if constexpr (DIR == kWeights) {
    bm = 128;
    g.I = N, g.J = K;
    g.nrt = (N + bm - 1) / bm, g.nct = (K + kCols - 1) / kCols;
    grid = (int64_t)(E + kXcds - 1) / kXcds * kXcds * g.nrt * g.nct;
  } else {
    bm = block % 128 == 0 ? 128 : block % 64 == 0 ? 64 : block % 32 == 0 ? 32 : 16;
    g.C = DIR == kForward ? K : N, g.J = DIR == kForward ? N : K;
    g.nrt = (int)(row_limit / bm), g.nct = (g.J + kCols - 1) / kCols;
    g.run = 8;
    grid = ((int64_t)g.nrt + kXcds * g.run - 1) / (kXcds * g.run) * g.run * kXcds * g.nct;
  }
  if (grid * kThreads > UINT32_MAX) return MRS_ERR_OVERFLOW;  // a launch has to have fewer than 2^32 threads
  void* params[] = {&g};
  return hipLaunchKernel(product_kernel<DIR>(dtype, out_dtype == MRS_DTYPE_F32, bm), dim3((unsigned)grid), dim3(kThreads),
                         params, 0, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? MRS_OK
             : MRS_ERR_LAUNCH;
}

}  // namespace

extern "C" int moe_grouped_gemm(const void* x, const void* w, int dtype, const int32_t* sorted_ids,
                                const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E, int K,
                                int N, int block, int x_rows, int y_dtype, void* y, void* stream) {
  return product<kForward>(x, w, dtype, sorted_ids, expert_of_block, num_post_pad, M, k, E, K, N, block, x_rows, y_dtype,
                           y, stream);
}

extern "C" int moe_grouped_gemm_dx(const void* dy, const void* w, int dtype, const int32_t* sorted_ids,
                                   const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E,
                                   int K, int N, int block, int dx_dtype, void* dx, void* stream) {
  return product<kRows>(dy, w, dtype, sorted_ids, expert_of_block, num_post_pad, M, k, E, K, N, block, MRS_X_SORTED,
                        dx_dtype, dx, stream);
}

extern "C" int moe_grouped_gemm_dw(const void* dy, const void* x, int dtype, const int32_t* sorted_ids,
                                   const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E,
                                   int K, int N, int block, int x_rows, int dw_dtype, void* dw, void* stream) {
  return product<kWeights>(dy, x, dtype, sorted_ids, expert_of_block, num_post_pad, M, k, E, K, N, block, x_rows,
                           dw_dtype, dw, stream);
}
