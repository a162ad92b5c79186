// Products grouped by expert in 16 bits, forward and backward, over the route-sort
// metadata, MI355X (gfx950, CDNA4, wave64).  Definitions: include/moe_experts.h.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "half.h"
#include "moe_experts.h"
#include "moe_route_sort.h"
#include "product_runs.h"

namespace {

// The three directions are one tiled product C[i, j] = sum_c A[i, c] B[j, c]:
//   kForward  i sorted rows, j = n, c = k: A = x (rows along c), B = w (rows along c)
//   kRows     i sorted rows, j = k, c = n: A = dy (rows along c), B = w (rows along j)
//   kWeights  i = n, j = k, c sorted rows of one expert: A = dy (rows along i), B = x
//             (rows along j)
// on v_mfma_f32_32x32x16, which sums 16 products in FP32.
//
// What bounds the large ones is what passes the L2s: 8.0 GB for y, 2.7 for dx and 1.8 for dw of
// the cases below, 6.4, 5.8 and 4.2 TB/s (a copy moves 4.9; the 256 MB cache answers a part).  y
// must move 5.3 GB, dx 0.95 and dw 0.5: XCDs and column tiles read operands again.  What bounds
// small and odd ones is how fast a compute unit takes operands out of its L2 (measured: 120 GB/s
// in whole 128-byte lines, 62 in halves of lines, 37 at odd addresses; LDS reads are 350 to 450).
// So: tiles as large as the registers hold where there are enough of them for every compute
// unit, and narrow ones where there are not; operands straight into LDS in whole lines where rows
// are whole chunks (steps of 64 along c); loads, LDS reads and matrix instructions of a wave
// interleaved; and what an expert's tiles share read from one L2 at about the same time.
//   8192 tokens, 896 experts, top-16, K 3584, N 768, blocks of 128: y in 1250 us; the bytes
//   that must move take 1075 at a copy's 4.9 TB/s (weights 4.9 GB); 577 TFLOP/s of routes
//   8192 tokens, 64 experts, top-8, the same K and N: dx in 440 to 470 us, dw in 400 to 440 (the
//   matrix units busy 43 to 50 % of it; an 8192^3 library product 1395 TFLOP/s, these 770 to 900)
enum Dir { kForward, kRows, kWeights };

struct GArgs {
  const uint16_t *a, *b;
  const int32_t *sid, *eob, *npp;
  void* out;
  int routes, k, E, block, sorted;
  int I, J, C;    // sizes of i, j, c (I: kWeights only; C: the others only)
  int row_limit;  // rows the metadata can hold: (max_rows / block) * block
  int nrt, nct;   // tiles of i (over all sorted rows, or of one expert), tiles of j
  int run;        // log2 of the row tiles of a run
  bool tiny;      // an operand's rows have fewer than eight values
};

// Operand tiles in LDS, in 16-byte chunks of eight values, a step of STEP values of c.
//
// Rows along c: the chunk at slot p of row r is p ^ ((r ^ (r >> 2)) & 3) (4 chunks a row)
// or p ^ (r & 7) ^ (r >> 3 & 1) (8 chunks), so that the 32 rows of an operand read hit
// distinct banks.
//
// Rows along the tile (one LDS row per c, W values wide): read by ds_read_b64_tr_b16,
// in which 16 lanes together read four rows of 16 values and each lane receives one
// column's four values.  Slot p of row c holds chunk p ^ (c & 3) << 2: the four rows
// that 32 lanes read 64 bytes of lie on distinct banks.
template <int STEP>
__device__ __forceinline__ int swz(int r, int p) {
  return STEP == 64 ? p ^ (r & 7) ^ ((r >> 3) & 1) : p ^ ((r ^ (r >> 2)) & 3);
}
__device__ __forceinline__ int swz_across(int c, int p) { return p ^ ((c & 3) << 2); }

typedef __attribute__((address_space(3))) char* lds_t;
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x2 read_turned(const char* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4*)(lds_t) const_cast<char*>(p)));
}

// Operand of v_mfma_*_32x32x16: lane l holds values 8 (l / 32) .. + 7 of c of row l mod
// 32; rows m0 .., c from 16 kk.
template <bool ACROSS, int W, int STEP>
__device__ __forceinline__ u32x4 operand(const u32x4* tile, int m0, int kk) {
  const int lane = threadIdx.x & 63;
  if constexpr (!ACROSS) {
    const int r = m0 + (lane & 31);
    return tile[r * (STEP / 8) + swz<STEP>(r, kk * 2 + (lane >> 5))];
  } else {
    static_assert(W >= 128, "chunks move within a row");
    const int c = kk * 16 + (lane >> 5) * 8 + ((lane & 15) >> 2);
    const int m = m0 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4;
    const char* p = reinterpret_cast<const char*>(tile + c * (W / 8) + swz_across(c, m / 8)) + (m & 4) * 2;
    const u32x2 lo = read_turned(p), hi = read_turned(p + 4 * (W / 8) * 16);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  }
}

// 16 bytes a lane from memory into LDS, lane l's at dst + 16 l.  Written out because
// the compiler waits for all such loads before any LDS read that it cannot tell from
// their targets, which leaves none in flight; the loop below counts them itself.  No
// register is written but m0: a reserved one, which the compiler sets right before an
// instruction that reads it, and refuses to take as clobbered.
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

// The blocks [first, last) of [0, n) that are expert e's: the first ones whose expert is
// at least e and at least e + 1, by two 64-ary searches side by side (the experts of used
// blocks ascend).
__device__ __forceinline__ void segment(const int32_t* eob, int n, int e, int& first, int& last) {
  const int lane = threadIdx.x & 63;
  int lo[2] = {0, 0}, len[2] = {n, n};  // the answers lie in [lo, lo + len]
  while (len[0] > 0 || len[1] > 0) {
    bool less[2];
    int step[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      step[i] = (len[i] + 63) / 64;
      less[i] = lane * step[i] < len[i] && eob[lo[i] + lane * step[i]] < e + i;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = __builtin_popcountll(__ballot(less[i]));  // probes 0 .. c - 1 are less
      const int from = c == 0 ? 0 : (c - 1) * step[i] + 1;
      lo[i] += from;
      len[i] = c == 0 ? 0 : min(step[i] - 1, len[i] - from);
    }
  }
  first = lo[0];
  last = lo[1];
}

// Workgroup h goes to XCD h mod 8.  Runs of consecutive row tiles (run_of) go to the XCDs
// in turn, the column tiles of a row tile one after another.  kWeights: an expert's column tiles
// go to the XCDs in turn with all their row tiles, so that large experts are everyone's (whole
// experts in turn 541 us, so 435).
constexpr int kRowsAhead = 4096;  // rows of an expert whose sources are kept in LDS at once (kWeights)

// A tile of BM x BN results by NW waves, in steps of STEP values of c, S stages of LDS.
template <int BM_, int BN_, int NW_, int STEP_, int S_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, NW = NW_, STEP = STEP_, S = S_;
  static constexpr int TR = BM < 32 ? 32 : BM;   // rows that are multiplied
  static constexpr int WI = BM >= 256 ? 4 : BM >= 128 ? 2 : 1, WJ = NW / WI;  // waves along i and j
  static constexpr int FM = TR / WI / 32, FN = BN / WJ / 32;  // operands of a wave
  static constexpr int kThreads = NW * 64;
  // workgroups of a compute unit by their LDS (160 KB), and so waves of a SIMD
  static constexpr int kPerSimd = NW < 4 ? 1 : (NW == 4 && (TR + BN) * STEP * 2 * S <= 76 << 10 ? 2 : 1) * NW / 4;
};

template <int DIR, typename P>
struct Ring {
  u32x4 a[P::S][P::TR * P::STEP / 8], b[P::S][P::BN * P::STEP / 8];
  int32_t row[DIR == kWeights ? kRowsAhead + 4 * P::STEP : P::TR];
  int32_t steps[P::NW];
};

// DIRECT: the operands' rows are whole 16-byte chunks at multiples of 16 bytes, and go
// from memory into LDS; otherwise through registers.
template <typename H, int DIR, typename P, bool F32, bool DIRECT>
__global__ __launch_bounds__(P::kThreads, P::kPerSimd) void k_product(GArgs g) {
  constexpr bool kAcrossA = DIR == kWeights, kAcrossB = DIR != kForward;
  constexpr int BM = P::BM, BN = P::BN, TR = P::TR, S = P::S, kStep = P::STEP, kThreads = P::kThreads;
  constexpr int WJ = P::WJ, FM = P::FM, FN = P::FN, kWaves = P::NW;
  constexpr int kChunks = kStep / 8;
  constexpr int AT = TR * kChunks;  // chunks of a stage of A
  constexpr int AP = (AT + kThreads - 1) / kThreads, BP = BN * kChunks / kThreads;  // of a thread
  constexpr int L = AP + BP;      // loads of a thread and stage
  constexpr int KK = kStep / 16;  // matrix instructions' steps of a stage
  __shared__ Ring<DIR, P> l;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int npp = min(*g.npp, g.row_limit);

  const int wi = wv / WJ * FM * 32, wj = wv % WJ * FN * 32;  // this wave's part of the tile
  int i0, j0, e, c_first = 0, c_end;  // the tile, its expert, the range of c
  uint64_t has = ~0ull;               // this wave's rows that hold a slot
  bool any = true;                    // some row of the tile does
  if constexpr (DIR == kWeights) {
    const int h = blockIdx.x, x = h % kXcds, q = h / kXcds, u = q / g.nrt * kXcds + x;
    e = u / g.nct;
    if (e >= g.E) return;
    i0 = q % g.nrt * BM, j0 = u % g.nct * BN;
    int first, last;
    segment(g.eob, max(npp, 0) / g.block, e, first, last);
    c_first = first * g.block, c_end = last * g.block;
  } else {
    const int h = blockIdx.x, x = h % kXcds, j = h / kXcds, i = j / g.nct;
    const int rt = (i >> g.run << 3 | x) << g.run | (i & ((1 << g.run) - 1));
    if (rt >= g.nrt) return;
    i0 = rt * BM, j0 = j % g.nct * BN;
    // asked for together, before any is looked at
    e = g.eob[i0 / g.block];
    const int s = tid < BM ? g.sid[i0 + tid] : -1;
    if (i0 + BM > npp || e < 0 || e >= g.E) return;  // npp is a multiple of block and BM divides block
    c_end = g.C;
    if (tid < TR) {
      const bool ok = s >= 0 && s < g.routes;
      l.row[tid] = !ok ? -1 : (DIR == kForward && !g.sorted) ? s / g.k : i0 + tid;
    }
    __syncthreads();
    has = __ballot(lane < FM * 32 && l.row[wi + lane % (FM * 32)] >= 0);
    any = __ballot(l.row[lane % TR] >= 0 || l.row[(lane + 64) % TR] >= 0) != 0;
  }
  e = __builtin_amdgcn_readfirstlane(e);

  // Sources of this thread's chunks p: slot tid + p * kThreads of a stage.
  // Rows along c: row sr + p * 64, chunk sc.  Across: c = tid / W + p * S, chunk by swz_across.
  constexpr int kRowStep = kThreads / kChunks;
  const int sr = tid / kChunks, sc = swz<kStep>(sr, tid % kChunks) * 8;
  constexpr int WA = TR / 8, SA = kThreads / WA, WB = BN / 8, SB = kThreads / WB;
  const int ia = i0 + swz_across(tid / WA, tid % WA) * 8, jb = j0 + swz_across(tid / WB, tid % WB) * 8;
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
    for (int p = 0; p < BP; ++p) pb[p] = g.b + ((int64_t)e * g.C + tid / WB + p * SB) * g.J;
  }

  const uint32_t lds_a = (uint32_t)(uintptr_t)(lds_t)(char*)l.a + (uint32_t)wv * 1024;
  const uint32_t lds_b = (uint32_t)(uintptr_t)(lds_t)(char*)l.b + (uint32_t)wv * 1024;
  const void* const zeros = &kZeros;
  // kWeights: the sources of a step's rows, -1 for none; the same for both operands, whose
  // tiles are equally wide
  static_assert(DIR != kWeights || WA == WB, "one map of rows");
  constexpr int RP = DIR != kWeights ? 1 : AP;
  auto find = [&](int (&to)[RP], int t) {
    if constexpr (DIR == kWeights) {
#pragma unroll
      for (int p = 0; p < AP; ++p) to[p] = l.row[t * kStep + tid / WA + p * SA];
    }
  };
  // Chunks whose rows run across the tile: the last chunk of a row ends with it, and so
  // do the results that come of it (out_of below).
  const int i_at = min(ia, g.I - 8), j_at = min(jb, g.J - 8);
  // Chunks along c: where a row ends inside step t its last chunks are read as its last
  // eight values, and moved down when they have arrived.
  auto along = [&](int t) {
    const int c0 = t * kStep;
    return DIRECT || c0 + kStep <= c_end ? c0 : min(c0 + sc, c_end - 8) - sc;
  };
  auto past = [&](int t) { return t * kStep + kStep <= c_end ? 0 : max(t * kStep + sc + 8 - c_end, 0); };
  auto chunk_a = [&](int t, int p, const int (&rows)[RP]) {
    if constexpr (!kAcrossA) return pa[p] + along(t);
    else return g.a + (int64_t)(c_first + t * kStep + tid / WA + p * SA) * g.I + i_at;
  };
  auto chunk_b = [&](int t, int p, const int (&rows)[RP]) {
    if constexpr (DIR == kForward) return pb[p] + along(t);
    else if constexpr (DIR == kRows) return pb[p] + (int64_t)t * kStep * g.J + j_at;
    else return g.b + (int64_t)max(rows[p], 0) * g.J + j_at;
  };
  // Whether a chunk's row of c (or, along c and straight into LDS, the chunk) exists.
  auto has_a = [&](int t, int p, const int (&rows)[RP]) {
    return kAcrossA ? rows[kAcrossA ? p : 0] >= 0 : !DIRECT || t * kStep + sc < c_end;
  };
  auto has_b = [&](int t, int p, const int (&rows)[RP]) {
    return DIR == kForward ? !DIRECT || t * kStep + sc < c_end
           : DIR == kRows  ? t * kStep + tid / WB + p * SB < c_end
                           : rows[DIR != kWeights ? 0 : p] >= 0;
  };
  // A part of step t of c, a KK-th (all of it where kPart is KK), into stage `buf` of LDS.
  auto issue = [&](int t, int buf, const int (&rows)[RP], auto part) {
    constexpr int kPart = decltype(part)::value;
    auto mine = [](int q) { return kPart == KK || q * KK / L == kPart; };
#pragma unroll
    for (int p = 0; p < AP; ++p) {
      if (!mine(p) || (AT % kThreads != 0 && tid + p * kThreads >= AT)) continue;
      const uint16_t* src = chunk_a(t, p, rows);
      load_lds(has_a(t, p, rows) ? src : zeros, lds_a + (buf * AT + p * kThreads) * 16);
    }
#pragma unroll
    for (int p = 0; p < BP; ++p) {
      if (!mine(AP + p)) continue;
      const uint16_t* src = chunk_b(t, p, rows);
      load_lds(has_b(t, p, rows) ? src : zeros, lds_b + (buf * BN * kChunks + p * kThreads) * 16);
    }
  };
  // Step t of c asked for into registers, and from there into stage `buf`.  Rows of fewer
  // than eight values (TINY) are loaded for themselves, one by one.
  struct Staged {
    u32x4 a[AP], b[BP];
    int rows[RP];
  };
  typedef const __attribute__((address_space(1))) u32x4_any* any_t;  // a choice of pointers keeps the address space
  auto fetch = [&](int t, Staged& r, auto tiny) {
    constexpr bool kTiny = decltype(tiny)::value;
#pragma unroll
    for (int p = 0; p < AP; ++p) {
      if (AT % kThreads != 0 && tid + p * kThreads >= AT) continue;
      if constexpr (kTiny) {
        const uint16_t* src = kAcrossA ? chunk_a(t, p, r.rows) - i_at + ia : pa[p] + t * kStep;
        r.a[p] = load8(src, !has_a(t, p, r.rows) ? 0 : kAcrossA ? g.I - ia : c_end - t * kStep - sc);
      } else {
        const any_t src = (any_t)(const u32x4_any*)chunk_a(t, p, r.rows);
        r.a[p] = *(has_a(t, p, r.rows) ? src : (any_t)(const u32x4_any*)&kZeros);
      }
    }
#pragma unroll
    for (int p = 0; p < BP; ++p) {
      if constexpr (kTiny) {
        const uint16_t* src = kAcrossB ? chunk_b(t, p, r.rows) - j_at + jb : pb[p] + t * kStep;
        r.b[p] = load8(src, !has_b(t, p, r.rows) ? 0 : kAcrossB ? g.J - jb : c_end - t * kStep - sc);
      } else {
        const any_t src = (any_t)(const u32x4_any*)chunk_b(t, p, r.rows);
        r.b[p] = *(has_b(t, p, r.rows) ? src : (any_t)(const u32x4_any*)&kZeros);
      }
    }
  };
  auto store = [&](int t, int buf, Staged& r, auto tiny) {
    if (!decltype(tiny)::value && DIR != kWeights && t * kStep + kStep > c_end) {
#pragma unroll
      for (int p = 0; p < AP; ++p) r.a[p] = drop(r.a[p], past(t));
      if constexpr (DIR == kForward) {
#pragma unroll
        for (int p = 0; p < BP; ++p) r.b[p] = drop(r.b[p], past(t));
      }
    }
#pragma unroll
    for (int p = 0; p < AP; ++p)
      if (AT % kThreads == 0 || tid + p * kThreads < AT) l.a[buf][tid + p * kThreads] = r.a[p];
#pragma unroll
    for (int p = 0; p < BP; ++p) l.b[buf][tid + p * kThreads] = r.b[p];
  };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
  struct Operands {
    u32x4 a[FM], b[FN];
  };
  auto read_one = [&](Operands& f, int buf, int kk, int q) {  // those of B first
    if (q < FN) f.b[q] = operand<kAcrossB, BN, kStep>(l.b[buf], wj + q * 32, kk);
    else f.a[q - FN] = operand<kAcrossA, TR, kStep>(l.a[buf], wi + (q - FN) * 32, kk);
  };
  auto multiply_one = [&](const Operands& f, int q) {
    acc[q / FN][q % FN] = H::mfma32(f.b[q % FN], f.a[q / FN], acc[q / FN][q % FN]);
  };
  auto next = [](int buf) { return buf + 1 == S ? 0 : buf + 1; };
  auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
  typedef std::integral_constant<int, KK> All;
  // Steps 0 .. n - 1 of c, all operands straight into LDS.  S - 1 stages are in flight; a
  // step past the last asks for zeros, so that every wait is for the same number.  The
  // matrix instructions of a k-step are interleaved with the reads of the next one's
  // operands and with a part of a stage's loads (left to itself the compiler reads the
  // operands right before their use).  A step has one barrier: past it the next stage
  // has arrived, and the stage read before is free.
  auto run_direct = [&](int n, auto parts) {
    // the leading parts of 32 rows of this wave that are multiplied: one without a slot is
    // not, and a wave without any only loads
    constexpr int kParts = decltype(parts)::value;
    constexpr bool kActive = kParts > 0;
    constexpr int kReads = kParts + FN, kMul = kActive ? kParts * FN : FN;
    Operands f[2];
    int rows[RP];
    // this wave's loads of S - 2 stages may be in flight
    auto wait_stage = [&] {
      if (AT < kThreads && wv >= AT / 64) wait_loads<(S - 2) * BP>();  // it loads no part of A
      else wait_loads<(S - 2) * L>();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) {
      find(rows, s);
      issue(s, s, rows, All());
    }
    find(rows, S - 1);
    wait_stage();
    barrier();
    int buf = 0, last = S - 1;  // the stages of step t and of step t + S - 1
    issue(S - 1, last, rows, std::integral_constant<int, 0>());
    if constexpr (kActive) {
#pragma unroll
      for (int q = 0; q < kReads; ++q) read_one(f[0], 0, 0, q);
    }
    for (int t = 0; t < n; ++t) {
      int ahead[RP];
      auto go = [&](auto kc) {
        constexpr int kk = decltype(kc)::value;
        constexpr int kAt = kk == KK - 1 && kMul > 1 ? 1 : 0;  // instructions before the reads
        fence();
#pragma unroll
        for (int q = 0; q < kMul; ++q) {
          if (kk == KK - 1 && q == kAt) {
            wait_stage();
            barrier();
            last = buf, buf = next(buf);
          }
          if (q == kAt) {
            if constexpr (kk == 0) find(ahead, t + S);
#pragma unroll
            for (int r = 0; r < (kReads + 1) / 2; ++r)
              if constexpr (kActive) read_one(f[(kk + 1) & 1], buf, (kk + 1) % KK, r);
          }
          if (kActive && q == (kAt + 1 < kMul ? kAt + 1 : kAt)) {
#pragma unroll
            for (int r = (kReads + 1) / 2; r < kReads; ++r) read_one(f[(kk + 1) & 1], buf, (kk + 1) % KK, r);
          }
          if constexpr (kActive) multiply_one(f[kk & 1], q);
          fence();
          if (q == (kMul > 2 ? 2 : kMul - 1)) {
            if constexpr (kk == KK - 1) {
#pragma unroll
              for (int r = 0; r < RP; ++r) rows[r] = ahead[r];
              issue(t + S, last, rows, std::integral_constant<int, 0>());
            } else {
              issue(t + S - 1, last, rows, std::integral_constant<int, kk + 1>());
            }
            fence();
          }
        }
      };
      go(std::integral_constant<int, 0>());
      go(std::integral_constant<int, 1>());
      if constexpr (KK == 4) {
        go(std::integral_constant<int, 2>());
        go(std::integral_constant<int, 3>());
      }
    }
    wait_loads<0>();
  };
  // Through registers, two steps in flight: a step is stored into LDS when it is its turn,
  // and the one after the next asked for.
  auto run_staged = [&](int n, bool active, auto tiny) {
    Staged r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      find(r[i].rows, i);
      fetch(i, r[i], tiny);
    }
    int buf = 0;
    auto step = [&](int t, Staged& q) {
      store(t, buf, q, tiny);
      find(q.rows, t + 2);
      barrier();
      fetch(t + 2, q, tiny);
      if (active) {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          Operands f;
#pragma unroll
          for (int x = 0; x < FM + FN; ++x) read_one(f, buf, kk, x);
#pragma unroll
          for (int x = 0; x < FM * FN; ++x) multiply_one(f, x);
        }
      }
      buf = next(buf);
    };
    for (int t = 0; t < n; t += 2) {  // a step past the last adds zeros
      step(t, r[0]);
      step(t + 1, r[1]);
    }
  };
  auto run = [&](int n, bool active) {
    if constexpr (DIRECT) {
      if (!active) run_direct(n, std::integral_constant<int, 0>());
      else if (FM == 2 && has >> 32 == 0) run_direct(n, std::integral_constant<int, 1>());
      else run_direct(n, std::integral_constant<int, FM>());
    } else {
      if (g.tiny) run_staged(n, active, std::true_type());  // rows of fewer than eight values
      else run_staged(n, active, std::false_type());
    }
    barrier();  // the stages and rows are free
  };
  if constexpr (DIR == kWeights) {
    const int end = c_end;
    for (int c = c_first; c < end; c += kRowsAhead) {
      const int n = min(end - c, kRowsAhead), whole = (n + kStep - 1) / kStep * kStep;
      int used = 0;  // steps up to the last row with a slot: an expert's padding comes last
      for (int r = tid; r < whole + 4 * kStep; r += kThreads) {
        const int s = r < n ? g.sid[c + r] : -1;
        const bool ok = s >= 0 && s < g.routes;
        l.row[r] = !ok ? -1 : g.sorted ? c + r : s / g.k;
        if (ok) used = r / kStep + 1;
      }
#pragma unroll
      for (int d = 1; d < 64; d *= 2) used = max(used, __shfl_xor(used, d));
      if (lane == 0) l.steps[wv] = used;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWaves; ++w) used = max(used, l.steps[w]);
      used = __builtin_amdgcn_readfirstlane(used);
      c_first = c;
      run(used, true);
    }
  } else {
    if (any) run((c_end + kStep - 1) / kStep, has != 0);  // a tile of padding reads nothing
  }

  // Result register v of lane l: column (of j) 8 (v / 4) + 4 (l / 32) + v mod 4, row (of i)
  // l mod 32.  A wave turns 32 rows at a time, and of FP32 half of its columns, in its part
  // of the LDS into whole chunks of 16 bytes of the output's rows.
  constexpr int JP = F32 && FN > 1 ? FN / 2 : FN;
  constexpr int kSize = F32 ? 4 : 2, kRow = JP * 32 * kSize, kPad = kRow + 16;  // bytes of a row in LDS
  static_assert(kWaves * 32 * kPad <= (int)(sizeof(l.a) + sizeof(l.b)), "the results fit");
  char* stage = reinterpret_cast<char*>(&l) + wv * 32 * kPad;
  const int64_t base = DIR == kWeights ? (int64_t)e * g.I : 0;
  // Where a row or column of the tile is stored, -1 for nowhere.  Of a chunk of eight that
  // passes the edge and was read as the last eight, all eight are: those before its own
  // place are stored twice, the same.
  auto out_of = [&](int at, int size) {
    const int first = at & ~7;
    if (DIRECT || g.tiny) return at < size ? at : -1;
    return first < size ? at - max(first + 8 - size, 0) : -1;
  };
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m0 = wi + i * 32;
    const bool ok = has >> (i * 32 + (lane & 31)) & 1;
#pragma unroll
    for (int j1 = 0; j1 < FN; j1 += JP) {
#pragma unroll
      for (int j = 0; j < JP; ++j)
#pragma unroll
        for (int v = 0; v < 16; v += 4) {
          char* at = stage + (lane & 31) * kPad + (j * 32 + 8 * (v / 4) + 4 * (lane >> 5)) * kSize;
          const f32x16& r = acc[i][j1 + j];
          f32x4 o = {r[v], r[v + 1], r[v + 2], r[v + 3]};
          if (!ok) o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (F32) *reinterpret_cast<f32x4*>(at) = o;
          else *reinterpret_cast<u32x2*>(at) = u32x2{H::pack(o[0], o[1]), H::pack(o[2], o[3])};
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int q = 0; q < 32 * kRow / 1024; ++q) {
        const int r = (q * 64 + lane) / (kRow / 16), c = (q * 64 + lane) % (kRow / 16);
        const int m = DIR == kWeights ? out_of(i0 + m0 + r, g.I) : m0 + r < BM ? i0 + m0 + r : -1;
        // rows of kForward and kRows are one of B's for each j, or one chunk for eight
        const int j = j0 + wj + j1 * 32 + c * (16 / kSize);
        const int n = DIR == kForward ? (j < g.J ? j : -1) : out_of(j, g.J);
        if (m >= 0 && n >= 0) {
          const u32x4 o = *reinterpret_cast<const u32x4*>(stage + r * kPad + c * 16);
          const int64_t at = (base + m) * g.J + n;
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
}

constexpr int kCols = 256;

// Tiles of each direction by their rows (us; kernels of 4 waves and up to 76 KB of LDS run
// two to a compute unit).
//   kForward, 128 rows: 8 waves, steps of 64 (whole lines) 1285 for the case above, 4 waves
//     and steps of 32 1506; 384 columns 1391 to 1412; fewer rows: steps of 64 in place of 32
//     445 for 486 (64 tokens of 896 experts, blocks of 16), 327 for 408 (2048 tokens of 256,
//     top-8, blocks of 64); seven stages of steps of 32: 22.6 for 18.7 (777 tokens of 24)
//   kRows: B runs across, in whole lines at any step: 128 rows by 4 waves and steps of 32
//     485, by 8 waves and steps of 64 512, pairs of blocks as tiles of 256 x 256 506 (the
//     case above; experts that share a pair take two passes); through registers they use all
//     256 and keep 8 (FP32 results) or 20 bytes a lane in scratch
//   kWeights: 256 x 256 by 8 waves 440, 128 x 256 by 8 waves 480, 128 x 128 487 (the case
//     above); 512 tokens of 896 experts 955, 1213, 1122
//   kWeights through registers: 128 x 128 by 8 waves 21.3 (777 tokens of 24 experts, K 1000,
//     N 397), by 4 waves 26.3, 128 x 256 24.0, 256 x 256 34 (it spills)
template <int DIR, int BM, int BN>
struct ShapeOf;
template <>
struct ShapeOf<kForward, 128, kCols> : Shape<128, kCols, 8, 64, 3> {};
template <>
struct ShapeOf<kForward, 64, kCols> : Shape<64, kCols, 4, 64, 3> {};
template <>
struct ShapeOf<kForward, 32, kCols> : Shape<32, kCols, 4, 64, 3> {};
template <>
struct ShapeOf<kForward, 16, kCols> : Shape<16, kCols, 4, 64, 3> {};
template <>
struct ShapeOf<kRows, 128, kCols> : Shape<128, kCols, 4, 32, 3> {};
template <>
struct ShapeOf<kRows, 64, kCols> : Shape<64, kCols, 4, 32, 3> {};
template <>
struct ShapeOf<kRows, 32, kCols> : Shape<32, kCols, 4, 32, 4> {};
template <>
struct ShapeOf<kRows, 16, kCols> : Shape<16, kCols, 4, 32, 4> {};
template <>
struct ShapeOf<kWeights, 256, kCols> : Shape<256, kCols, 8, 32, 3> {};  // straight into LDS
template <>
struct ShapeOf<kWeights, 128, 128> : Shape<128, 128, 8, 32, 3> {};  // through registers, or few of them
// Narrow ones, for few workgroups
constexpr int narrow(int dir) { return dir == kForward ? 64 : 128; }
template <int BM>
struct ShapeOf<kForward, BM, narrow(kForward)> : Shape<BM, narrow(kForward), 2, 64, 4> {};
template <int BM>
struct ShapeOf<kRows, BM, narrow(kRows)> : Shape<BM, narrow(kRows), 4, 32, 4> {};

struct Launch {
  const void* kernel;
  int threads;
};

template <typename H, int DIR, bool F32, bool DIRECT, int BM, int BN>
Launch launch_of() {
  typedef ShapeOf<DIR, BM, BN> P;
  return {reinterpret_cast<const void*>(k_product<H, DIR, P, F32, DIRECT>), P::kThreads};
}

template <typename H, int DIR, bool F32, bool DIRECT, int BN>
Launch product_kernel(int bm) {
  switch (bm) {
    case 64: return launch_of<H, DIR, F32, DIRECT, 64, BN>();
    case 32: return launch_of<H, DIR, F32, DIRECT, 32, BN>();
    default: return launch_of<H, DIR, F32, DIRECT, 16, BN>();
  }
}

template <typename H, int DIR, bool F32, bool DIRECT>
Launch product_kernel(int bm, int bn) {
  if constexpr (DIR == kWeights) {
    if constexpr (DIRECT) {
      if (bm == 256) return launch_of<H, DIR, F32, DIRECT, 256, kCols>();
    }
    return launch_of<H, DIR, F32, DIRECT, 128, 128>();
  } else {
    if (bn != kCols) return product_kernel<H, DIR, F32, DIRECT, narrow(DIR)>(bm);
    if (bm == 128) return launch_of<H, DIR, F32, DIRECT, 128, kCols>();
    return product_kernel<H, DIR, F32, DIRECT, kCols>(bm);
  }
}

template <typename H, int DIR>
Launch product_kernel(bool f32, int bm, int bn, bool direct) {
  if (direct) return f32 ? product_kernel<H, DIR, true, true>(bm, bn) : product_kernel<H, DIR, false, true>(bm, bn);
  return f32 ? product_kernel<H, DIR, true, false>(bm, bn) : product_kernel<H, DIR, false, false>(bm, bn);
}

constexpr int kMaxCols = 1 << 20;

template <int DIR>
int product(const void* a, const void* b, int dtype, const int32_t* sid, const int32_t* eob, const int32_t* npp, int M,
            int k, int E, int K, int N, int block, int x_rows, int out_dtype, void* out, void* stream, int tile = 0) {
  const int rows = tile & ~MRS_TILE_NARROW;
  if (M < 0 || k < 1 || k > 64 || E < 1 || E > 4096 || K < 1 || K > kMaxCols || N < 1 || N > kMaxCols || block < 16 ||
      block % 16 != 0 || (dtype != MRS_DTYPE_BF16 && dtype != MRS_DTYPE_F16) ||
      (out_dtype != dtype && out_dtype != MRS_DTYPE_F32) || (x_rows != MRS_X_TOKENS && x_rows != MRS_X_SORTED) ||
      (tile != 0 && ((rows != 16 && rows != 32 && rows != 64 && (rows != 128 || tile != rows)) || block % rows != 0)))
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
  // lengths of the operands' rows
  const int la = DIR == kForward ? K : N, lb = K;
  g.tiny = la < 8 || lb < 8;
  const bool direct = la % 8 == 0 && aligned_to(a, 16) && lb % 8 == 0 && aligned_to(b, 16);
  const bool f32 = out_dtype == MRS_DTYPE_F32;
  int bm, bn = kCols;
  int64_t grid;
  if constexpr (DIR == kWeights) {
    const int64_t large = (int64_t)E * ((N + 255) / 256) * ((K + 255) / 256);
    // us, 256 x 256 / 128 x 128: 200 tokens of 16 experts, top-2, K 512, N 256 (32 large tiles) 7.7 /
    // 5.0; 32 of 16, K 768, N 512 (96) 7.9 / 7.0; 777 of 24, top-6, K 1000, N 400 (192) 15.5 / 19.6
    bm = direct && large >= 128 ? 256 : 128;
    if (bm == 128) bn = 128;
    g.I = N, g.J = K;
    g.nrt = (N + bm - 1) / bm, g.nct = (K + bn - 1) / bn;
    grid = ((int64_t)E * g.nct + kXcds - 1) / kXcds * kXcds * g.nrt;
  } else {
    g.C = DIR == kForward ? K : N, g.J = DIR == kForward ? N : K;
    // The largest tile that divides the block, but 64 rows where fewer than 128 workgroups would
    // come of it, and then narrow tiles where they are fewer still.  kForward: fewer than 256 where
    // an expert is one tile, so that its weights are read once either way; where it is more, tiles
    // of 64 rows and whole chunks, if the narrow ones run at once.  us, wide / narrow, kForward:
    // 300 tokens of 8 experts, top-2, K 2048, N 1024 21.5 / 13.6; 400 of 8, N 1280 26.7 / 16.1; 200
    // of 4, N 4096 29.0 / 23.7; 2000 of 2, top-1, N 1024 20.2 / 26.9; 512 of 8, K 3584, N 1536 (three
    // row tiles of 24 columns on an XCD) 47.4 / 67.4, and where their average just fits, but not an
    // uneven XCD, K 2048, N 1280 28.0 / 33.8; 200 of 24, top-6, K 1000, N 400 12.1 / 8.7; 48 of 31,
    // top-3, K 1713, N 109 30.8 / 12.9; one of 896, top-16, K 3584, N 768 26.2 / 18.0, four of them
    // 59.8 / 53.4; 777 of 24 (192 workgroups) 17.1 / 23; rows that are no whole chunks, 1000 of 8,
    // top-2, K 1001, N 515 26.1 / 15.5.  kRows: 200 of 24 8.0 / 7.1, one of 896 (224) 16.1 / 16.5, 48
    // of 31 (217) 9.1 / 11.1.  Narrow tiles of few rows an expert are of 32 rows (48 of 31 16.7, so
    // 12.9; 100 rows an expert 12.7 for 13.6), and kForward takes them for any number of such
    // experts where operands go through registers, which are slower to fill (256 of 256, top-8, K
    // 1203, N 515 102 / 76; 40 of 120, top-14, K 1209, N 676 58 / 39; 64 of 896, top-16, K 1001, N
    // 397 129 / 111; with whole chunks, K 2048, N 768, 512 of 128 97 / 99).
    bm = block % 128 == 0 ? 128 : block % 64 == 0 ? 64 : block % 32 == 0 ? 32 : 16;
    const int64_t routes = (int64_t)M * k, used = routes < E ? routes : E, average = (routes + used - 1) / used;
    auto tiles = [&] { return used * ((average + bm - 1) / bm) * ((g.J + bn - 1) / bn); };
    while (bm > 64 && tiles() < 128) bm /= 2;
    const bool short_rows = DIR == kForward && !direct && average <= 32;
    const bool fits = row_limit * ((g.J + 63) / 64) < 1 << 28;  // more threads than wide ones, fewer than 2^32
    auto few = [&] {
      if (DIR == kForward && average <= bm) return tiles() < 256;
      if (DIR == kRows || !direct || bm < 64) return tiles() < 128;
      return tiles() <= 128 && at_once(used, average, bm, block, (g.J + narrow(DIR) - 1) / narrow(DIR));
    };
    if (fits && (short_rows || (bm <= 64 && few()))) {
      bn = narrow(DIR);
      if (bm > 32 && average <= 32) bm = 32;
    }
    if (tile != 0) bm = rows, bn = tile == rows ? kCols : narrow(DIR);
    g.nrt = (int)(row_limit / bm), g.nct = (g.J + bn - 1) / bn;
    g.run = run_of(used, average, bm, block);
    const int64_t group = kXcds << g.run;
    grid = (g.nrt + group - 1) / group * group * g.nct;
  }
  const Launch p = dtype == MRS_DTYPE_BF16 ? product_kernel<BF16, DIR>(f32, bm, bn, direct)
                                           : product_kernel<FP16, DIR>(f32, bm, bn, direct);
  if (DIR != kWeights && grid * p.threads > UINT32_MAX)  // the shortest runs have the fewest tiles past the last
    g.run = 0, grid = (g.nrt + kXcds - 1) / kXcds * (int64_t)kXcds * g.nct;
  if (grid * p.threads > UINT32_MAX) return MRS_ERR_OVERFLOW;  // a launch has to have fewer than 2^32 threads
  void* params[] = {&g};
  return hipLaunchKernel(p.kernel, dim3((unsigned)grid), dim3(p.threads), params, 0,
                         reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? MRS_OK
             : MRS_ERR_LAUNCH;
}

}  // namespace

extern "C" int moe_grouped_gemm_ex(const void* x, const void* w, int dtype, const int32_t* sorted_ids,
                                   const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E,
                                   int K, int N, int block, int x_rows, int y_dtype, void* y, void* stream, int tile) {
  return product<kForward>(x, w, dtype, sorted_ids, expert_of_block, num_post_pad, M, k, E, K, N, block, x_rows, y_dtype,
                           y, stream, tile);
}

extern "C" int moe_grouped_gemm(const void* x, const void* w, int dtype, const int32_t* sorted_ids,
                                const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E, int K,
                                int N, int block, int x_rows, int y_dtype, void* y, void* stream) {
  return moe_grouped_gemm_ex(x, w, dtype, sorted_ids, expert_of_block, num_post_pad, M, k, E, K, N, block, x_rows,
                             y_dtype, y, stream, 0);
}

extern "C" int moe_grouped_gemm_dx_ex(const void* dy, const void* w, int dtype, const int32_t* sorted_ids,
                                      const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E,
                                      int K, int N, int block, int dx_dtype, void* dx, void* stream, int tile) {
  return product<kRows>(dy, w, dtype, sorted_ids, expert_of_block, num_post_pad, M, k, E, K, N, block, MRS_X_SORTED,
                        dx_dtype, dx, stream, tile);
}

extern "C" int moe_grouped_gemm_dx(const void* dy, const void* w, int dtype, const int32_t* sorted_ids,
                                   const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E,
                                   int K, int N, int block, int dx_dtype, void* dx, void* stream) {
  return moe_grouped_gemm_dx_ex(dy, w, dtype, sorted_ids, expert_of_block, num_post_pad, M, k, E, K, N, block, dx_dtype,
                                dx, stream, 0);
}

extern "C" int moe_grouped_gemm_dw(const void* dy, const void* x, int dtype, const int32_t* sorted_ids,
                                   const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k, int E,
                                   int K, int N, int block, int x_rows, int dw_dtype, void* dw, void* stream) {
  return product<kWeights>(dy, x, dtype, sorted_ids, expert_of_block, num_post_pad, M, k, E, K, N, block, x_rows,
                           dw_dtype, dw, stream);
}
