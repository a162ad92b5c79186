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
  const uint16_t *a, *b, *a_end, *b_end;
  const int32_t *sid, *eob, *npp;
  void* out;
  int routes, k, E, block, sorted;
  int I, J, C;    // sizes of i, j, c (I: kWeights only; C: the others only)
  int row_limit;  // rows the metadata can hold: (max_rows / block) * block
  int nrt, nct;   // tiles of i (over all sorted rows, or of one expert), tiles of j
  int run;        // consecutive row tiles of an XCD
};

constexpr int kThreads = 256, kWaves = 4;
constexpr int kStep = 32;  // of c

// Operand tiles in LDS, in 16-byte chunks of eight values.
//
// Rows along c: 4 chunks a row, the chunk at slot p of row r is p ^ ((r ^ (r >> 2)) & 3),
// so that the 32 rows of an operand read hit distinct banks.
//
// Rows along the tile (one LDS row per c, W values wide): read by ds_read_b64_tr_b16,
// in which 16 lanes together read four rows of 16 values and each lane receives one
// column's four values.  Slot p of row c holds chunk p ^ (c & 3) << 2: the four rows
// that 32 lanes read 64 bytes of lie on distinct banks.
__device__ __forceinline__ int swz(int r, int p) { return p ^ ((r ^ (r >> 2)) & 3); }
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
    return tile[r * (kStep / 8) + swz(r, kk * 2 + (lane >> 5))];
  } else {
    const int c = kk * 16 + (lane >> 5) * 8 + ((lane & 15) >> 2);
    const int m = m0 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
    const char* p = reinterpret_cast<const char*>(tile + c * (W / 8) + swz_across<W>(c, m / 8)) + (m & 4) * 2;
    const u32x2 lo = read_turned(p), hi = read_turned(p + 4 * (W / 8) * 16);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  }
}

// 16 bytes a lane from memory into LDS, lane l's at dst + 16 l.  Written out because
// the compiler waits for all such loads before any LDS read that it cannot tell from
// their targets, which leaves none in flight; the loop below counts them itself.  No
// register is written but m0, which the compiler keeps nothing in.
__device__ __forceinline__ void load_lds(const void* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(dst), "v"(src) : "memory");
}
// All but the last N of this wave's loads have arrived.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// This wave's LDS accesses are through, and every wave is here.
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ const u32x4 kZeros = {0u, 0u, 0u, 0u};

// Eight values at any element's address, zeros past the first n; `end` is the end of
// the matrix: a load that stays below it is made whole and its tail cleared.
__device__ __forceinline__ u32x4 load8_any(const uint16_t* p, int n, const uint16_t* end) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (n <= 0) return v;
  if (p + 8 > end) return load8(p, n);
  v = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = n >= 2 * i + 2 ? v[i] : n == 2 * i + 1 ? v[i] & 0xFFFFu : 0u;
  return v;
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
template <int BM>
constexpr int stages() {
  return BM < 64 ? 4 : 3;
}
constexpr int kRowsAhead = 1024;  // rows of an expert whose sources are kept in LDS at once (kWeights)

template <int DIR, int BM, int BN>
struct Ring {
  static constexpr int kRows = tile_rows<BM>();
  u32x4 a[stages<BM>()][kRows * kStep / 8], b[stages<BM>()][BN * kStep / 8];
  int32_t row[DIR == kWeights ? kRowsAhead : kRows];
};

// DA, DB: the operand's rows and chunks are whole and 16-byte aligned, and go from
// memory into LDS; otherwise through registers.
template <typename H, int DIR, int BM, int BN, bool F32, bool DA, bool DB>
__global__ __launch_bounds__(kThreads, 2) void k_product(GArgs g) {
  constexpr bool kAcrossA = DIR == kWeights, kAcrossB = DIR != kForward;
  constexpr int TR = tile_rows<BM>(), S = stages<BM>();
  constexpr int WI = BM >= 128 ? 2 : 1, WJ = kWaves / WI;  // waves along i and j
  constexpr int FM = TR / WI / 32, FN = BN / WJ / 32;
  constexpr int kChunks = kStep / 8;
  constexpr int AT = TR * kChunks;  // chunks of a stage of A
  constexpr int AP = (AT + kThreads - 1) / kThreads, BP = BN * kChunks / kThreads;  // of a thread
  constexpr int L = AP + BP;  // loads into LDS of a wave and stage
  __shared__ Ring<DIR, BM, BN> l;
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

  // Sources of this thread's chunks p: slot tid + p * kThreads of a stage.
  // Rows along c: row sr + p * 64, chunk sc.  Across: c = tid / W + p * S, chunk by swz_across.
  constexpr int kRowStep = kThreads / kChunks;
  const int sr = tid / kChunks, sc = swz(sr, tid % kChunks) * 8;
  constexpr int WA = TR / 8, SA = kThreads / WA, WB = BN / 8, SB = kThreads / WB;
  const int ia = i0 + swz_across<128>(tid / WA, tid % WA) * 8, jb = j0 + swz_across<BN>(tid / WB, tid % WB) * 8;
  const uint16_t* const end_a = g.a_end;
  const uint16_t* const end_b = g.b_end;
  const uint16_t *pa[kAcrossA ? 1 : AP], *pb[DIR == kWeights ? 1 : BP];
  if constexpr (!kAcrossA) {
#pragma unroll
    for (int p = 0; p < AP; ++p) {  // a padding row's chunks come from row 0 and its results are replaced
      const int r = sr + p * kRowStep;
      pa[p] = g.a + (int64_t)max(r < TR ? l.row[r] : 0, 0) * g.C + sc;
    }
  }
  if constexpr (DIR == kForward) {
#pragma unroll
    for (int p = 0; p < BP; ++p)  // columns past the last repeat it and are not stored
      pb[p] = g.b + ((int64_t)e * g.J + min(j0 + sr + p * kRowStep, g.J - 1)) * g.C + sc;
  } else if constexpr (DIR == kRows) {
#pragma unroll
    for (int p = 0; p < BP; ++p)
      pb[p] = g.b + ((int64_t)e * g.C + tid / WB + p * SB) * g.J + (DB ? min(jb, g.J - 8) : jb);
  }

  const uint32_t lds_a = (uint32_t)(uintptr_t)(lds_t)(char*)l.a + (uint32_t)wv * 1024;
  const uint32_t lds_b = (uint32_t)(uintptr_t)(lds_t)(char*)l.b + (uint32_t)wv * 1024;
  const void* const zeros = &kZeros;
  u32x4 ra[AP], rb[BP];

  // step t of c: into stage `buf` of LDS, or into registers
  auto issue = [&](int t, int buf) {
    const int c0 = t * kStep;  // kWeights: from the first of the rows in l.row
    if constexpr (!kAcrossA) {
#pragma unroll
      for (int p = 0; p < AP; ++p) {
        if (AT % kThreads == 0 || tid + p * kThreads < AT) {
          const uint16_t* src = pa[p] + c0;
          if constexpr (DA)
            load_lds(c0 + kStep <= c_end || c0 + sc < c_end ? src : zeros,
                     lds_a + (buf * AT + p * kThreads) * 16);
          else
            ra[p] = load8_any(src, c_end - c0 - sc, end_a);
        }
      }
    } else {
#pragma unroll
      for (int p = 0; p < AP; ++p) {
        const int c = c0 + tid / WA + p * SA;
        const bool ok = l.row[c] >= 0;
        const uint16_t* src = g.a + (int64_t)(c_first + c) * g.I + (DA ? min(ia, g.I - 8) : ia);
        if constexpr (DA) load_lds(ok ? src : zeros, lds_a + (buf * AT + p * kThreads) * 16);
        else ra[p] = load8_any(src, ok ? g.I - ia : 0, end_a);
      }
    }
#pragma unroll
    for (int p = 0; p < BP; ++p) {
      const uint32_t dst = lds_b + (buf * BN * kChunks + p * kThreads) * 16;
      if constexpr (DIR == kForward) {
        const uint16_t* src = pb[p] + c0;
        if constexpr (DB) load_lds(c0 + kStep <= c_end || c0 + sc < c_end ? src : zeros, dst);
        else rb[p] = load8_any(src, c_end - c0 - sc, end_b);
      } else if constexpr (DIR == kRows) {
        const uint16_t* src = pb[p] + (int64_t)c0 * g.J;
        const bool ok = c0 + tid / WB + p * SB < c_end;
        if constexpr (DB) load_lds(c0 + kStep <= c_end || ok ? src : zeros, dst);
        else rb[p] = load8_any(src, ok ? g.J - jb : 0, end_b);
      } else {
        const int row = l.row[c0 + tid / WB + p * SB];
        const uint16_t* src = g.b + (int64_t)max(row, 0) * g.J + (DB ? min(jb, g.J - 8) : jb);
        if constexpr (DB) load_lds(row >= 0 ? src : zeros, dst);
        else rb[p] = load8_any(src, row >= 0 ? g.J - jb : 0, end_b);
      }
    }
  };
  auto store = [&](int buf) {
    if constexpr (!DA) {
#pragma unroll
      for (int p = 0; p < AP; ++p)
        if (AT % kThreads == 0 || tid + p * kThreads < AT) l.a[buf][tid + p * kThreads] = ra[p];
    }
    if constexpr (!DB) {
#pragma unroll
      for (int p = 0; p < BP; ++p) l.b[buf][tid + p * kThreads] = rb[p];
    }
  };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
  const int wi = wv / WJ * FM * 32, wj = wv % WJ * FN * 32;
  auto multiply = [&](int buf) {
#pragma unroll
    for (int kk = 0; kk < kStep / 16; ++kk) {
      u32x4 fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[i] = operand<kAcrossA, TR>(l.a[buf], wi + i * 32, kk);
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[j] = operand<kAcrossB, BN>(l.b[buf], wj + j * 32, kk);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = H::mfma32(fb[j], fa[i], acc[i][j]);
    }
  };
  auto next = [](int buf) { return buf + 1 == S ? 0 : buf + 1; };
  // Steps 0 .. n - 1 of c.  All operands straight into LDS: S - 1 stages in flight, one
  // barrier a step, past which the stage multiplied before is free.  Through registers:
  // a step's are stored when the next one's have been asked for.
  auto run = [&](int n) {
    if constexpr (DA && DB) {
#pragma unroll
      for (int s = 0; s < S - 1; ++s)
        if (s < n) issue(s, s);
      int buf = 0, free = S - 1;
      for (int t = 0; t < n; ++t) {
        const int newer = min(S - 2, n - 1 - t);  // stages asked for after this one
        if (newer == 0) wait_loads<0>();
        else if (AT < kThreads && wv >= AT / 64) newer == 1 ? wait_loads<BP>() : wait_loads<2 * BP>();  // no part of A
        else newer == 1 ? wait_loads<L>() : wait_loads<2 * L>();
        barrier();
        if (t + S - 1 < n) issue(t + S - 1, free);
        multiply(buf);
        buf = next(buf), free = next(free);
      }
    } else {
      issue(0, 0);
      int buf = 0;
      for (int t = 0; t < n; ++t) {
        store(buf);
        wait_loads<0>();
        barrier();
        if (t + 1 < n) issue(t + 1, next(buf));
        multiply(buf);
        buf = next(buf);
      }
    }
    barrier();  // the stages and rows are free
  };
  if constexpr (DIR == kWeights) {
    const int end = c_end;
    for (int c = c_first; c < end; c += kRowsAhead) {
      const int n = min(end - c, kRowsAhead), whole = (n + kStep - 1) / kStep * kStep;
      for (int r = tid; r < whole; r += kThreads) {
        const int s = r < n ? g.sid[c + r] : -1;
        const bool ok = s >= 0 && s < g.routes;
        l.row[r] = !ok ? -1 : g.sorted ? c + r : s / g.k;
      }
      __syncthreads();
      c_first = c;
      run(whole / kStep);
    }
  } else {
    run((c_end + kStep - 1) / kStep);
  }

  // Result register v of lane l: column (of j) 8 (v / 4) + 4 (l / 32) + v mod 4, row (of i)
  // l mod 32.  A wave turns 32 rows at a time in its part of the LDS into whole chunks of
  // 16 bytes of the output's rows.
  constexpr int kSize = F32 ? 4 : 2, kRow = FN * 32 * kSize, kPad = kRow + 16;  // bytes of a row in LDS
  static_assert(kWaves * 32 * kPad <= (int)(sizeof(l.a) + sizeof(l.b)), "the results fit");
  char* stage = reinterpret_cast<char*>(&l) + wv * 32 * kPad;
  const int64_t base = DIR == kWeights ? (int64_t)e * g.I : 0;
  const int rows = DIR == kWeights ? g.I - i0 : BM;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m0 = wi + i * 32, m = m0 + (lane & 31);
    const bool ok = m >= 64 ? has[1] >> (m - 64) & 1 : has[0] >> m & 1;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; v += 4) {
        char* at = stage + (lane & 31) * kPad + (j * 32 + 8 * (v / 4) + 4 * (lane >> 5)) * kSize;
        f32x4 o = {acc[i][j][v], acc[i][j][v + 1], acc[i][j][v + 2], acc[i][j][v + 3]};
        if (!ok) o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (F32) *reinterpret_cast<f32x4*>(at) = o;
        else *reinterpret_cast<u32x2*>(at) = u32x2{H::pack(o[0], o[1]), H::pack(o[2], o[3])};
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int q = 0; q < 32 * kRow / 1024; ++q) {
      const int r = (q * 64 + lane) / (kRow / 16), c = (q * 64 + lane) % (kRow / 16);
      const int n = j0 + wj + c * (16 / kSize);
      if (m0 + r < rows && n < g.J) {
        const u32x4 o = *reinterpret_cast<const u32x4*>(stage + r * kPad + c * 16);
        const int64_t at = (base + i0 + m0 + r) * g.J + n;
        if constexpr (F32) {
          float* out = static_cast<float*>(g.out) + at;
          if (n + 4 <= g.J) {
            __builtin_nontemporal_store(o, reinterpret_cast<u32x4_f32*>(out));
          } else {
#pragma unroll
            for (int x = 0; x < 3; ++x)
              if (n + x < g.J) out[x] = __uint_as_float(o[x]);
          }
        } else {
          store8(static_cast<uint16_t*>(g.out) + at, o, g.J - n);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

constexpr int kCols = 256;

template <typename H, int DIR, bool F32, bool DA, bool DB>
const void* product_kernel(int bm) {
  if constexpr (DIR == kWeights) {
    return reinterpret_cast<const void*>(k_product<H, DIR, 128, kCols, F32, DA, DB>);
  } else {
    switch (bm) {
      case 128: return reinterpret_cast<const void*>(k_product<H, DIR, 128, kCols, F32, DA, DB>);
      case 64: return reinterpret_cast<const void*>(k_product<H, DIR, 64, kCols, F32, DA, DB>);
      case 32: return reinterpret_cast<const void*>(k_product<H, DIR, 32, kCols, F32, DA, DB>);
      default: return reinterpret_cast<const void*>(k_product<H, DIR, 16, kCols, F32, DA, DB>);
    }
  }
}

template <typename H, int DIR, bool F32>
const void* product_kernel(int bm, bool da, bool db) {
  if (da && db) return product_kernel<H, DIR, F32, true, true>(bm);
  // rows along c have one length in both operands
  if constexpr (DIR != kForward) {
    if (da) return product_kernel<H, DIR, F32, true, false>(bm);
    if (db) return product_kernel<H, DIR, F32, false, true>(bm);
  }
  return product_kernel<H, DIR, F32, false, false>(bm);
}

template <int DIR>
const void* product_kernel(int dtype, bool f32, int bm, bool da, bool db) {
  if (dtype == MRS_DTYPE_BF16)
    return f32 ? product_kernel<BF16, DIR, true>(bm, da, db) : product_kernel<BF16, DIR, false>(bm, da, db);
  return f32 ? product_kernel<FP16, DIR, true>(bm, da, db) : product_kernel<FP16, DIR, false>(bm, da, db);
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
  // lengths of the operands' rows and their numbers
  const int la = DIR == kForward ? K : N, lb = K;
  const int64_t na = DIR == kForward && !g.sorted ? M : max_rows;
  const int64_t nb = DIR != kWeights ? (int64_t)E * N : g.sorted ? max_rows : M;
  g.a_end = g.a + na * la, g.b_end = g.b + nb * lb;
  const bool da = la % 8 == 0 && aligned_to(a, 16), db = lb % 8 == 0 && aligned_to(b, 16);
  void* params[] = {&g};
  return hipLaunchKernel(product_kernel<DIR>(dtype, out_dtype == MRS_DTYPE_F32, bm, da, db), dim3((unsigned)grid), dim3(kThreads),
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
