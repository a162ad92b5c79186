// 4-bit microscaled rows and their grouped product, MI355X (gfx950, CDNA4,
// wave64).  Definitions and argument contracts: include/moe_mxfp4.h.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_mxfp4.h"
#include "moe_route_sort.h"

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// ------------------------------------------------------------ quantisation
//
// A thread takes eight consecutive columns, so four neighbouring lanes hold
// one block of 32: its largest magnitude is two quad permutes of the integer
// maximum of the bit patterns (which orders infinities and NaN above every
// number).  The scale's exponent field is the maximum's less two, the values
// are multiplied by the exact power of two and v_cvt_scalef32_pk_fp4_f32
// rounds two at a time.

struct QArgs {
  const void* x;
  uint8_t* codes;
  uint8_t* scales;
  void* values;
  int64_t rows, stride, groups;  // groups: eights of columns, rows * gpr
  int K, gpr;                    // gpr: groups per row, Kp / 8
  uint32_t gpr_mul;              // ceil(2^32 / gpr): exact below 2^17 + 2^8
  uint64_t gpr_mul64;            // floor(2^64 / gpr) + 1: exact below 2^49
};

template <int DT>
struct Elem;
template <>
struct Elem<MRS_DTYPE_F32> {
  typedef float T;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<MRS_DTYPE_BF16> {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t put(float v) { return (uint16_t)(__float_as_uint(v) >> 16); }
};
template <>
struct Elem<MRS_DTYPE_F16> {
  typedef _Float16 T;
  static __device__ __forceinline__ float get(_Float16 v) { return (float)v; }
  static __device__ __forceinline__ _Float16 put(float v) { return (_Float16)v; }
};

constexpr int kQThreads = 256;

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  // quad_perm [1,0,3,2], then [2,3,0,1]
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
}

// Eight values as stored.  Rows need no more alignment than their elements: the
// wide global accesses accept that.
template <typename T>
union Eight {
  T v[8];
  u32x4 q[sizeof(T) / 2];
};
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Every lane of a quad belongs to the same row (gpr is a multiple of 16) and all
// of them run.
template <int DT, bool VALUES>
__global__ __launch_bounds__(kQThreads) void k_quantize(QArgs a) {
  typedef Elem<DT> El;
  typedef typename El::T T;
  const int64_t g0 = (int64_t)blockIdx.x * kQThreads;
  const int64_t row0 = (int64_t)__umul64hi((uint64_t)g0, a.gpr_mul64);  // g0 / gpr
  const uint32_t in = (uint32_t)(g0 - row0 * a.gpr) + threadIdx.x;
  const uint32_t dr = __umulhi(in, a.gpr_mul);  // in / gpr
  const int64_t row = row0 + dr;
  const int g = (int)(in - dr * (uint32_t)a.gpr), c0 = g * 8;
  const bool live = row < a.rows;
  const T* src = static_cast<const T*>(a.x) + row * a.stride + c0;
  Eight<T> raw;
  if (live && c0 + 8 <= a.K) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) raw.q[i] = reinterpret_cast<const u32x4_any*>(src)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) raw.v[i] = live && c0 + i < a.K ? src[i] : T(0);
  }
  float v[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = El::get(raw.v[i]);
    top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  }
  top = quad_max(top);
  const uint32_t field = top >> 23;  // 0 for zeros and subnormals
  const bool bad = field == 255u;
  const uint32_t X = bad ? 255u : (uint32_t)max((int)field - 2, 0);
  const float inv = __uint_as_float((254u - X) << 23);  // 2^(127 - X); X <= 252 where it is used
  uint32_t code = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float p = bad ? 0.0f : v[2 * i] * inv, q = bad ? 0.0f : v[2 * i + 1] * inv;
    switch (i) {  // the byte to write is an immediate
      case 0: code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, p, q, 1.0f, 0); break;
      case 1: code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, p, q, 1.0f, 1); break;
      case 2: code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, p, q, 1.0f, 2); break;
      default: code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, p, q, 1.0f, 3); break;
    }
  }
  if (!live) return;
  reinterpret_cast<uint32_t*>(a.codes)[row * a.gpr + g] = code;
  if ((g & 3) == 0) a.scales[(row * a.gpr + g) >> 2] = (uint8_t)X;
  if constexpr (VALUES) {
    f32x2 d[4];
    d[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 0);
    d[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 1);
    d[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 2);
    d[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 3);
    T* dst = static_cast<T*>(a.values) + row * a.K + c0;
    Eight<T> o;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o.v[i] = El::put(bad ? __uint_as_float(0x7FC00000u) : ldexpf(d[i / 2][i % 2], (int)X - 127));
    if (c0 + 8 <= a.K) {
      // one whole store past the L2; FP32's two half-line stores are put together there
      // (131072 x 768 BF16 76 -> 63 us, 20011 x 1001 FP32 27 -> 31)
      if constexpr (sizeof(T) == 2) {
        __builtin_nontemporal_store(o.q[0], reinterpret_cast<u32x4_any*>(dst));
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) reinterpret_cast<u32x4_any*>(dst)[i] = o.q[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + i < a.K) dst[i] = o.v[i];
    }
  }
}

// A launch has to have fewer than 2^32 threads, and each takes one group.
constexpr int64_t kQLaunch = int64_t(1) << 31;  // groups of one launch, in whole rows

template <int DT>
const void* quant_kernel(bool values) {
  return values ? reinterpret_cast<const void*>(k_quantize<DT, true>)
                : reinterpret_cast<const void*>(k_quantize<DT, false>);
}

// --------------------------------------------------------- grouped product

struct PArgs {
  const uint8_t *xc, *xs, *wc, *ws;
  const int32_t *sid, *eob, *npp;
  void* y;
  int M, k, E, K, N, block, sorted;
  int row_limit;  // rows the metadata can hold: (max_rows / block) * block
  int nrt, ntn;   // row tiles, column tiles
  int run;        // consecutive row tiles of an XCD
  bool large;     // the weights are larger than the 256 MB cache in front of the memory
};

// Workgroup h goes to XCD h mod 8; runs of `run` consecutive row tiles go to the
// XCDs in turn, the column tiles of a row tile one after another, so an expert's
// row tiles read its weights, and a row tile's column tiles its rows, from one L2
// at about the same time.
constexpr int kXcds = 8;
__device__ __forceinline__ void tile_of(int h, int run, int ntn, int& rt, int& ct) {
  const int x = h % kXcds, j = h / kXcds, i = j / ntn;
  rt = (i / run * kXcds + x) * run + i % run;
  ct = j % ntn;
}

// Few rows an expert: pairs of a padding block (G row tiles) and a column tile go
// to the XCDs in turn, kPairs of them together, first row tiles first.  The later
// row tiles are often padding only: pair by pair they fell to every G-th compute
// unit and left it idle (one token, blocks of 32: 11.6 us).
constexpr int kPairs = 16;
__device__ __forceinline__ bool tile_of_block(int h, int G, int ntn, int nrt, int& rt, int& ct) {
  const int x = h % kXcds, j = h / kXcds;
  const int u = (j / (G * kPairs) * kPairs + j % kPairs) * kXcds + x;
  rt = u / ntn * G + j / kPairs % G;
  ct = u % ntn;
  return rt < nrt;
}

__device__ __forceinline__ void put_y(float* y, float v) { *y = v; }
// FP32 to BF16, round to nearest even; NaN stays NaN.
__device__ __forceinline__ void put_y(uint16_t* y, float v) {
  const uint32_t u = __float_as_uint(v);
  const uint32_t r = u + 0x7FFFu + ((u >> 16) & 1u);
  *y = v != v ? (uint16_t)0x7FC0u : (uint16_t)(r >> 16);
}

// Whether 16-byte chunks of y's rows are whole and aligned.
template <typename Y>
__device__ __forceinline__ bool wide_rows(const PArgs& a) {
  return a.N % (16 / sizeof(Y)) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
}

// Zeros in a workgroup's tile of BM rows x BN columns, 256 threads.
template <typename Y, int BM, int BN>
__device__ __forceinline__ void zero_tile(const PArgs& a, int r0, int n0) {
  const int tid = threadIdx.x;
  Y* y = static_cast<Y*>(a.y) + (size_t)r0 * a.N + n0;
  if (wide_rows<Y>(a)) {
    constexpr int kChunk = 16 / sizeof(Y), kRow = BN / kChunk;  // values of a chunk, chunks of a row
    const int c = tid % kRow * kChunk;
    if (n0 + c < a.N)
      for (int r = tid / kRow; r < BM; r += 256 / kRow)
        __builtin_nontemporal_store(u32x4{0u, 0u, 0u, 0u}, reinterpret_cast<u32x4*>(y + (size_t)r * a.N + c));
  } else {
    const int c = tid % BN;
    if (n0 + c < a.N)
      for (int r = tid / BN; r < BM; r += 256 / BN) put_y(y + (size_t)r * a.N + c, 0.0f);
  }
}

__device__ __forceinline__ i32x8 frag(u32x4 q) {
  const i32x4 v = __builtin_bit_cast(i32x4, q);
  return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}

// Few rows an expert: tiles of 16 rows x 16 FN columns, the four waves of a
// workgroup taking every fourth step of 128 columns and adding up in LDS at the
// end.  Bound by the weights' bytes: each lane reads its 16-byte chunks of W
// straight into the matrix operand's registers (v_mfma_scale_f32_16x16x128:
// lane l holds columns 32 (l / 16) .. + 31 of row l mod 16, which is one chunk
// and one scale byte), U steps in flight at a time, and nothing goes through
// LDS but the partial sums.  Padding rows load nothing.  896 experts, top-16, K =
// 3584, N = 768, blocks of 32: one token in 8.8 us, 24 MB at 2.7 TB/s, of which 3.4
// us pass with a single step (the launch, the metadata, one round trip).  Eight
// steps in flight measured best (64 tokens 203 us, six or ten 220 us).
constexpr int kRowsDeep = 8;
// Fewer tiles of 32 columns than this: tiles of 16 (one token, 384 tiles: 9.6 and
// 11.7 us; two tokens, 768 tiles: 17.2 and 16.0 us).
constexpr int kRowsNarrow = 512;

template <typename Y, int FN>
__global__ __launch_bounds__(256) void k_product_rows(PArgs a) {
  constexpr int U = kRowsDeep;
  __shared__ f32x4 part[4][FN][64];
  int rt, ct;
  if (!tile_of_block((int)blockIdx.x, a.block / 16, a.ntn, a.nrt, rt, ct)) return;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  const int r0 = rt * 16, n0 = ct * 16 * FN;
  const int npp = min(*a.npp, a.row_limit);
  const int e = a.eob[r0 / a.block];
  const int s = a.sid[r0 + r16];
  if (r0 >= npp || e < 0 || e >= a.E) return;
  const bool ok = s >= 0 && s < a.M * a.k;
  const uint32_t rows = (uint32_t)__ballot(ok) & 0xFFFFu;
  if (!rows) {  // padding only
    zero_tile<Y, 16, 16 * FN>(a, r0, n0);
    return;
  }
  f32x4 acc[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) acc[j] = f32x4{};
  {
    const size_t kb = (size_t)a.K / 2, ks = (size_t)a.K / 32;
    const size_t xr = ok ? (size_t)(a.sorted ? r0 + r16 : s / a.k) : 0;
    const uint8_t* xc = a.xc + xr * kb + q * 16;
    const uint8_t* xs = a.xs + xr * ks;
    const uint8_t *wc[FN], *ws[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const size_t n = (size_t)e * a.N + min(n0 + j * 16 + r16, a.N - 1);
      wc[j] = a.wc + n * kb + q * 16;
      ws[j] = a.ws + n * ks;
    }
    const int steps = a.K / 128, wave = __builtin_amdgcn_readfirstlane(wv);
    u32x4 xq[U], wq[U][FN];
    int xe[U], we[U][FN];
    auto load = [&](int u, int t) {
      xq[u] = u32x4{0u, 0u, 0u, 0u};
      xe[u] = 0;
      if (ok) {
        xq[u] = *reinterpret_cast<const u32x4*>(xc + t * 64);
        xe[u] = *reinterpret_cast<const int*>(xs + t * 4);
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        wq[u][j] = *reinterpret_cast<const u32x4*>(wc[j] + t * 64);
        we[u][j] = *reinterpret_cast<const int*>(ws[j] + t * 4);
      }
    };
    auto multiply = [&](int u) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            frag(xq[u]), frag(wq[u][j]), acc[j], 4, 4, 0, (int)((uint32_t)xe[u] >> (8 * q)), 0,
            (int)((uint32_t)we[u][j] >> (8 * q)));
    };
    int t = wave;
    for (; t + 4 * (U - 1) < steps; t += 4 * U) {
#pragma unroll
      for (int u = 0; u < U; ++u) load(u, t + 4 * u);
#pragma unroll
      for (int u = 0; u < U; ++u) multiply(u);
    }
    const int left = (steps - t + 3) / 4;  // of this wave, fewer than U
#pragma unroll
    for (int u = 0; u < U - 1; ++u)
      if (u < left) load(u, t + 4 * u);
#pragma unroll
    for (int u = 0; u < U - 1; ++u)
      if (u < left) multiply(u);
  }
#pragma unroll
  for (int j = 0; j < FN; ++j) part[wv][j][lane] = acc[j];
  __syncthreads();
  // result register i of lane l: row 4 (l / 16) + i, column l mod 16
  const float* p = reinterpret_cast<const float*>(part);
#pragma unroll
  for (int i = 0; i < FN; ++i) {
    const int o = i * 256 + threadIdx.x, row = o / (16 * FN), c = o % (16 * FN);
    const int at = ((c / 16) * 64 + (row / 4) * 16 + c % 16) * 4 + row % 4;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += p[w * FN * 256 + at];
    if (n0 + c < a.N)
      put_y(static_cast<Y*>(a.y) + (size_t)(r0 + row) * a.N + n0 + c, (rows >> row) & 1u ? v : 0.0f);
  }
}

// Tiles of BM rows x 256 columns, four waves of 64 columns each
// (v_mfma_scale_f32_32x32x64: lane l holds columns 32 (l / 32) .. + 31 of row
// l mod 32).  Steps of 256 columns, 128 bytes a row: the x rows are shared by the
// waves, each wave's weight rows are its own.  Both are read eight lanes to a
// row and turned in LDS (16-byte chunks XOR-swizzled, so that the 32 rows of an
// operand read hit distinct banks), the next step's into registers while the
// present one is multiplied.  Reading the weights straight into operand
// registers, every lane another row, kept the address unit busy 87 % of the time
// and bounded the kernel.  8192 tokens, 896 experts, top-16, K = 3584, N = 768 in
// 435 us: 1.6 GB that must move at 3.7 TB/s; with the experts' rows read again
// from the L2's misses and y written, 2.2 GB at 5.0 TB/s (a 2 GiB copy: 4.9), which
// bounds it now (without the multiplications it takes 410 us).  64 tokens of the
// same experts in blocks of 16: 901 MB of weights in 150 us, 6.0 TB/s.
constexpr int kFN = 2, kNW = 4;  // 32-column operands a wave, waves
constexpr int kCols = kNW * kFN * 32, kTileThreads = kNW * 64;

__device__ __forceinline__ int swz(int r, int c) { return r * 8 + (c ^ (r & 7) ^ ((r >> 3) & 1)); }

struct alignas(8) Scale8 {
  uint32_t lo, hi;
};

// Scale words of a run of kScaleSteps steps (64 bytes a row), staged into LDS at
// once: fetched step by step, a row's line left the L2 between two steps and came
// from memory for each of them (2.1 GB read in place of 1.7 on 8192 tokens x 896
// experts).  Row r keeps the pair of step t at slot t ^ ((r / 4) mod 8), so that
// the 32 rows of an operand lie on distinct banks.
constexpr int kScaleSteps = 8;
__device__ __forceinline__ int scale_slot(int r, int t) { return r * kScaleSteps + (t ^ ((r >> 2) & 7)); }

// ROWS rows' words into LDS (slot order above), straight from memory: lane l of
// the wave's instruction i (the wave's q-th) fills word i * 64 + l, `src(row)` is
// the row's first word of the run, words past `left` repeat the last one and are
// not used.
template <int ROWS, typename F>
__device__ __forceinline__ void stage_scales(Scale8* dst, int left, F src) {
  constexpr int kEach = ROWS * kScaleSteps * 2 / 64 / kNW;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll 2
  for (int q = 0; q < kEach; ++q) {
    const int i = wv * kEach + q, o = i * 64 + lane, r = o / (2 * kScaleSteps);
    const int t = ((o / 2) % kScaleSteps) ^ ((r >> 2) & 7), w = min(2 * t + (o & 1), left - 1);
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src(r) + w * 4),
                                     (__attribute__((address_space(3))) void*)(reinterpret_cast<uint32_t*>(dst) + i * 64),
                                     4, 0, 0);
  }
}

// Rows that a tile of BM multiplies: one of 16 fills half an operand, the other
// half repeats row 0 of x and is not stored.
constexpr int tile_rows(int BM) { return BM < 32 ? 32 : BM; }
// Steps in flight while one is multiplied: two where the registers allow it (2048
// tokens, 256 experts, top-8, K = 3584, N = 768, blocks of 64: 109 us with one, 92
// with two; tiles of 128 rows spill with two, tiles of 32 are slower with three, 223
// against 213).
constexpr int deep_of(int BM) { return BM < 128 ? 2 : 1; }

// Whether weights that one row tile alone reads are loaded past the L2 (another
// copy of the loop, which tiles of 64 rows and more have no registers for).
template <int BM>
constexpr bool kOnce = BM <= 32;

template <int BM>
struct Tile {
  static constexpr int kRows = tile_rows(BM);
  u32x4 x[kRows * 8], w[kCols * 8];
  Scale8 sx[kRows * kScaleSteps], sw[kCols * kScaleSteps];
  uint32_t row[kRows];  // row of x
};

constexpr int kWP = kFN * 32 * 8 / 64;  // weight chunks a lane stages in a step
typedef u32x4 WeightRegs[kWP];

// The rows of W that this wave stages: lane l takes chunk l mod 8 of rows l / 8, + 8, ...
struct Weights {
  const uint8_t *codes, *scales;  // of the tile's first column
  int row, last;                  // this lane's first row, the last row that exists
  uint32_t kb;                    // bytes of a row
  // o: byte of the row.  ONCE: no other row tile reads these weights, and the L2 need
  // not keep them (896 experts, blocks of 16: 64 tokens 177 -> 165 us, 512 tokens 251 ->
  // 241; so loaded where row tiles share them, 2048 tokens and 256 experts 176 -> 220; nor
  // where all experts' fit the cache in front of the memory, which may have them from
  // the call before: 50 MB 13.6 -> 14.7).
  template <bool ONCE>
  __device__ __forceinline__ void load(WeightRegs& q, int o) const {
#pragma unroll
    for (int p = 0; p < kWP; ++p) {
      int r = row + p * 8;
      asm volatile("" : "+v"(r));  // opaque: eight row addresses kept over the loop spill
      const u32x4* at = reinterpret_cast<const u32x4*>(codes + ((uint32_t)min(r, last) * kb + (uint32_t)o));
      q[p] = ONCE ? __builtin_nontemporal_load(at) : *at;
    }
  }
};

__device__ __forceinline__ void wait_memory() { __builtin_amdgcn_s_waitcnt(0x0F70); }  // vmcnt(0)

// `has`: a bit for each row that holds a route; `live`: the leading 32-row parts
// of the tile that have one
template <typename Y, int BM, bool ONCE>
__device__ __forceinline__ void tile_body(const PArgs& a, int r0, int n0, const uint64_t (&has)[2], int live,
                                          const Weights& w, WeightRegs (&wr)[deep_of(BM)], Tile<BM>& l) {
  constexpr int kDeep = deep_of(BM);
  constexpr int TR = tile_rows(BM), FM = TR / 32;
  constexpr int XP = TR * 8 / kTileThreads;  // x chunks a thread stages in a step
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int lr = lane & 31, lh = lane >> 5;
  const size_t kb = (size_t)a.K / 2, ks = (size_t)a.K / 32;
  const int steps = (a.K + 255) / 256;
  const bool half = a.K % 256 != 0;  // the last step has 128 columns

  // Padding rows read row 0: each row's result is its own, and theirs is
  // replaced by zero.  Past K, in the second half of a last step of 128 columns,
  // the first half is read again with both scale words zero: 2^-254 times any
  // codes vanishes in FP32.
  const int c16 = tid % 8 * 16, back = tid % 8 >= 4 ? 64 : 0;
  auto at = [&](int t) { return t * 128 + c16 - (half && t == steps - 1 ? back : 0); };
  const uint8_t* xsrc[XP];
#pragma unroll
  for (int p = 0; p < XP; ++p) xsrc[p] = a.xc + (size_t)l.row[(tid + p * kTileThreads) / 8] * kb;
  typedef u32x4 RowRegs[XP];
  RowRegs xr[kDeep];
  auto load = [&](RowRegs& x, WeightRegs& q, int t) {
    w.template load<ONCE>(q, at(t));
#pragma unroll
    for (int p = 0; p < XP; ++p) x[p] = *reinterpret_cast<const u32x4*>(xsrc[p] + at(t));
  };
  auto store = [&](const RowRegs& x, const WeightRegs& q) {
#pragma unroll
    for (int p = 0; p < XP; ++p) l.x[swz((tid + p * kTileThreads) / 8, tid % 8)] = x[p];
#pragma unroll
    for (int p = 0; p < kWP; ++p) l.w[swz(wv * kFN * 32 + lane / 8 + p * 8, tid % 8)] = q[p];
  };
  auto load_scales = [&](int t, bool weights) {
    // opaque, or the addresses of the runs after the first are made ahead of the
    // loop and kept (100 registers spilled)
    uint32_t kv = (uint32_t)ks;
    asm volatile("" : "+s"(kv));
    const int left = (int)kv / 4 - t * 2;  // words left in a row
    stage_scales<TR>(l.sx, left, [&](int r) { return a.xs + (size_t)l.row[r] * kv + t * 8; });
    if (weights)
      stage_scales<kCols>(l.sw, left, [&](int r) { return w.scales + (size_t)min(r, w.last) * kv + t * 8; });
  };

#pragma unroll
  for (int p = 0; p < XP; ++p) xr[0][p] = *reinterpret_cast<const u32x4*>(xsrc[p] + at(0));
  load_scales(0, false);
  if constexpr (kDeep == 2) load(xr[1], wr[1], min(1, steps - 1));
  store(xr[0], wr[0]);
  wait_memory();  // the scales are in LDS
  __syncthreads();
  __builtin_amdgcn_sched_barrier(0);
  f32x16 acc[FM][kFN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < kFN; ++j) acc[i][j] = f32x16{};

  // step t, whose operands are in LDS: those of step t + kDeep go into the
  // registers that step t's have left
  auto step = [&](int t, RowRegs& x, WeightRegs& q) {
    if (t > 0 && t % kScaleSteps == 0) {  // past the last step's barrier
      load_scales(t, true);
      wait_memory();
      __syncthreads();
    }
    const uint32_t keep = half && t == steps - 1 ? 0u : ~0u;
    load(x, q, min(t + kDeep, steps - 1));
    // scale of columns 64 g + 32 lh ..: byte 2 (g mod 2) of the word g / 2 shifted by 8 lh
    Scale8 we[kFN];
#pragma unroll
    for (int j = 0; j < kFN; ++j) {
      we[j] = l.sw[scale_slot((wv * kFN + j) * 32 + lr, t % kScaleSteps)];
      we[j].lo >>= 8 * lh;
      we[j].hi = (we[j].hi & keep) >> (8 * lh);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // two groups of 64 columns
      i32x8 wf[kFN][2], xf[2];
      Scale8 xe;
      auto read = [&](int i) {
#pragma unroll
        for (int g = 0; g < 2; ++g) xf[g] = frag(l.x[swz(i * 32 + lr, 4 * h + 2 * g + lh)]);
        xe = l.sx[scale_slot(i * 32 + lr, t % kScaleSteps)];
      };
#pragma unroll
      for (int j = 0; j < kFN; ++j)
#pragma unroll
        for (int g = 0; g < 2; ++g) wf[j][g] = frag(l.w[swz((wv * kFN + j) * 32 + lr, 4 * h + 2 * g + lh)]);
      read(0);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const i32x8 x0 = xf[0], x1 = xf[1];
        const int xs = (int)((h == 0 ? xe.lo : xe.hi & keep) >> (8 * lh));
        if (i + 1 < FM) read(i + 1);
        if (i < live)
#pragma unroll
          for (int j = 0; j < kFN; ++j) {
            const int ws = (int)(h == 0 ? we[j].lo : we[j].hi);
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x0, wf[j][0], acc[i][j], 4, 4, 0, xs, 0, ws);
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x1, wf[j][1], acc[i][j], 4, 4, 2, xs, 2, ws);
          }
      }
    }
    __syncthreads();
  };
  int t = 0;
  if constexpr (kDeep == 2) {
    // no way out of the middle: with one, the compiler waits in every step for loads
    // that only the last one has in flight
    for (; t + 2 < steps; t += 2) {
      step(t, xr[0], wr[0]);
      store(xr[1], wr[1]);
      __syncthreads();
      step(t + 1, xr[1], wr[1]);
      store(xr[0], wr[0]);
      __syncthreads();
    }
    step(t, xr[0], wr[0]);
    if (t + 1 < steps) {
      store(xr[1], wr[1]);
      __syncthreads();
      step(t + 1, xr[1], wr[1]);
    }
  } else {
    for (;;) {
      step(t, xr[0], wr[0]);
      if (++t == steps) break;
      store(xr[0], wr[0]);
      __syncthreads();
    }
  }

  // Result register v of lane l: row 8 (v / 4) + 4 (l / 32) + v mod 4, column
  // l mod 32.  A wave turns its 32 x 64 results in its own part of the LDS (the
  // last barrier has passed, rows and scales are used up) into whole 16-byte
  // chunks of y's rows.
  constexpr int kRow = kFN * 32 * sizeof(Y), kPad = kRow + 16;  // bytes of a row in LDS
  static_assert(kNW * 32 * kPad <= (int)(sizeof(l.x) + sizeof(l.w)), "the results fit");
  const bool wide = wide_rows<Y>(a);
  char* stage = reinterpret_cast<char*>(&l) + wv * 32 * kPad;
  const int n1 = n0 + wv * kFN * 32;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const uint32_t rows = (uint32_t)(has[i / 2] >> (i % 2 * 32));
    Y* y = static_cast<Y*>(a.y) + (size_t)(r0 + i * 32) * a.N;
    if (wide) {
#pragma unroll
      for (int j = 0; j < kFN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int r = 8 * (v / 4) + 4 * lh + v % 4;
          const float o = (rows >> r) & 1u ? acc[i][j][v] : 0.0f;
          put_y(reinterpret_cast<Y*>(stage + r * kPad) + j * 32 + lr, o);
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int q = 0; q < 32 * kRow / 1024; ++q) {
        const int r = (q * 64 + lane) / (kRow / 16), c = (q * 64 + lane) % (kRow / 16);
        const int n = n1 + c * (16 / (int)sizeof(Y));
        const u32x4 o = *reinterpret_cast<const u32x4*>(stage + r * kPad + c * 16);
        // not kept in the L2, which the rows and weights need (8192 tokens, 896 experts:
        // 447 -> 435 us; 64 tokens, 256 experts, blocks of 128: 93.5 -> 87)
        if (n < a.N && (BM >= 32 || r < BM))
          __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(y + (size_t)r * a.N + n));
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    } else {
#pragma unroll
      for (int j = 0; j < kFN; ++j) {
        const int n = n1 + j * 32 + lr;
        if (n < a.N)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int r = 8 * (v / 4) + 4 * lh + v % 4;
            const float o = (rows >> r) & 1u ? acc[i][j][v] : 0.0f;
            if (BM >= 32 || r < BM) put_y(y + (size_t)r * a.N + n, o);
          }
      }
    }
  }
}

template <typename Y, int BM>
__global__ __launch_bounds__(kTileThreads, 2) void k_product_tile(PArgs a) {
  __shared__ Tile<BM> l;
  int rt, ct;
  tile_of((int)blockIdx.x, a.run, a.ntn, rt, ct);
  if (rt >= a.nrt) return;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int r0 = rt * BM, n0 = ct * kCols;
  const int npp = min(*a.npp, a.row_limit);
  const int blk = r0 / a.block, e = __builtin_amdgcn_readfirstlane(a.eob[blk]);
  // the only row tile of its expert?  A block of several tiles counts as shared.
  int before = e, after = e;
  if constexpr (kOnce<BM>) {
    before = blk > 0 ? a.eob[blk - 1] : -1;
    after = r0 + a.block < a.row_limit ? a.eob[blk + 1] : -1;
  }
  int s[2];  // slots of rows lane and 64 + lane, in every wave
#pragma unroll
  for (int i = 0; i < 2; ++i) s[i] = i * 64 + lane < BM ? a.sid[r0 + i * 64 + lane] : -1;
  if (r0 + BM > npp || e < 0 || e >= a.E) return;  // npp is a multiple of block and BM divides block
  bool ok[2];
  uint64_t has[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ok[i] = s[i] >= 0 && s[i] < a.M * a.k;
    has[i] = __ballot(ok[i]);
  }
  if (!(has[0] | has[1])) {  // padding only: no weights are read
    zero_tile<Y, BM, kCols>(a, r0, n0);
    return;
  }
  const size_t kb = (size_t)a.K / 2, ks = (size_t)a.K / 32;
  const Weights w{a.wc + ((size_t)e * a.N + n0) * kb, a.ws + ((size_t)e * a.N + n0) * ks,
                  wv * kFN * 32 + lane / 8, a.N - 1 - n0, (uint32_t)kb};
  WeightRegs wr[deep_of(BM)];
  const bool once = kOnce<BM> && a.large && BM == a.block && before != e && (r0 + BM >= npp || after != e);
  const int o0 = tid % 8 * 16 - (a.K == 128 && tid % 8 >= 4 ? 64 : 0);
  if (once) w.template load<kOnce<BM>>(wr[0], o0);
  else w.template load<false>(wr[0], o0);
  stage_scales<kCols>(l.sw, (int)ks / 4, [&](int r) { return w.scales + (size_t)min(r, w.last) * ks; });
  if (tid < l.kRows) {  // the first two waves, lane tid mod 64
    const bool mine = ok[wv & 1];
    const int slot = s[wv & 1];
    l.row[tid] = mine ? (a.sorted ? r0 + tid : slot / a.k) : 0;
  }
  __syncthreads();
  // a segment's routes come first: the last 32 rows that hold one bound the work
  int live = has[1] >> 32 ? 4 : has[1] ? 3 : has[0] >> 32 ? 2 : 1;
  // opaque: knowing that the first part is live the compiler merges its block
  // with the step's loads and spills inside the loop (1.5 ms in place of 0.45)
  asm volatile("" : "+s"(live));
  if (once) tile_body<Y, BM, kOnce<BM>>(a, r0, n0, has, live, w, wr, l);
  else tile_body<Y, BM, false>(a, r0, n0, has, live, w, wr, l);
}

template <typename Y>
const void* product_kernel(int bm, int bn) {
  if (bn == 16) return reinterpret_cast<const void*>(k_product_rows<Y, 1>);
  if (bn == 32) return reinterpret_cast<const void*>(k_product_rows<Y, 2>);
  switch (bm) {
    case 128: return reinterpret_cast<const void*>(k_product_tile<Y, 128>);
    case 64: return reinterpret_cast<const void*>(k_product_tile<Y, 64>);
    case 32: return reinterpret_cast<const void*>(k_product_tile<Y, 32>);
    default: return reinterpret_cast<const void*>(k_product_tile<Y, 16>);
  }
}

// Tile sizes from the expected load.  Strips are the weights' tiles of 256 columns
// over the experts that get a route; a workgroup of the tile kernel streams one.
// With few of them and few rows the rows kernel's smaller tiles fill the chip (us,
// rows kernel / tile kernel; K = 3584, N = 768, blocks of 32): 1 token of 896 experts,
// top-16, 48 strips 8.9 / 16.6; 2 tokens, 96 strips 14.5 / 18.0; 3 tokens, 144 strips
// 20.3 / 20.0.  It reads the weights again for every 16 rows: 8 experts, 24 strips, 16
// rows an expert 9.7 / 15.7, 64 rows 19.4 / 16.5.  And a block's row tiles that have
// padding only are workgroups too, 1 ns each, while the tile kernel's time is its
// steps': one token as above in blocks of 128 13.9 / 15.8, of 256 19.6 / 15.9; 64 experts,
// K = 2048, 2 tokens, top-8, blocks of 64 9.7 / 10.5, of 128 12.7 / 10.5; K = 1024, N = 512,
// 4 tokens, top-4, blocks of 64 5.9 / 7.6, of 256 13.0 / 7.6.
//
// The tile kernel takes the largest tile that divides the block (a part of 32 rows
// without a route costs no multiplications; 256 experts, K = 3584, blocks of 128, 64 /
// 128 / 192 rows an expert: tiles of 128 100 / 124 / 154 us, of 64 96 / 129 / 173, of 32
// 117 / 165 / 220), but none of 128 for fewer than 48 rows, of which most of the steps'
// loads would be padding's (16 rows 97 / 87 / 91; blocks of 256 107 / 100 / 98), and
// smaller ones where 128 workgroups would not come together (8 experts, 512 tokens:
// tiles of 32 8.2 us, 64 10.2, 128 14.1).  With 128 to 255 workgroups of the chosen tile the
// next smaller one is still 1 to 42 % faster, from 256 on they are level (us, tiles of 32
// / 64 / 128; 2 experts, K = 3584, N = 2048: 512 rows each 18.1 / 21.5 / 29.6, 1024 rows 24.4 /
// 22.1 / 30.8, 2048 rows 43.8 / 31.5 / 32.4; 24 experts, K = 1024, N = 396, 341 rows each 16.2 /
// 13.4 / 15.2; 64 experts, K = 3584, N = 396, 256 rows each 56.1 / 49.5 / 44.1).
//
// Runs of row tiles: eight or more for each XCD, so that none has much more than
// another (us with runs of 8 / with this rule: 2048 tokens, 64 experts, top-8 45.5 /
// 34.0; 8192 tokens, 8 experts, top-2, blocks of 256 53.6 / 47.9), powers of two up
// to 16 (8192 tokens, 896 experts: 428, runs of 23 446).  Whole blocks, or the
// tiles that have routes, the first of each block, fall to some of the XCDs only (64
// experts, K = 1024, 16 rows an expert, blocks of 128 12.8 / 10.0, of 256 22 / 11) and an
// expert's weights are read by all of them (8 experts, 250 rows each, blocks of 256 16.5
// / 13.8); but not those of fewer experts than XCDs with routes in most of a block's
// tiles, which would keep to a few XCDs (2 experts, blocks of 1024 34 / 21.5).
struct Shape {
  int bm, bn, run;
};
// `kernel`: one that the caller names in place of the rule's (run by the rule).
Shape shape_of(int64_t routes, int64_t used, int K, int N, int block, int kernel) {
  const int64_t cols = (N + kCols - 1) / kCols, strips = used * cols;
  int bm;
  switch (kernel) {
    case MRS_PRODUCT_ROWS_16: return {16, 16, 1};
    case MRS_PRODUCT_ROWS_32: return {16, 32, 1};
    case MRS_PRODUCT_TILE_16: bm = 16; break;
    case MRS_PRODUCT_TILE_32: bm = 32; break;
    case MRS_PRODUCT_TILE_64: bm = 64; break;
    case MRS_PRODUCT_TILE_128: bm = 128; break;
    default:
      if (strips < 192 && strips * routes <= 768 * used && strips * (block / 16) <= 160 + K / 16)
        return {16, used * ((N + 31) / 32) < kRowsNarrow ? 16 : 32, 1};
      bm = block % 128 == 0 && routes > 48 * used ? 128 : block % 64 == 0 ? 64 : block % 32 == 0 ? 32 : 16;
      while (strips < 192 && bm > 32 && routes / bm * cols < 128) bm /= 2;
  }
  const int64_t tiles = routes / bm + used / 2;  // an expert's last tile is half full
  int run = 1;
  while (run < 16 && run * 128 <= tiles) run *= 2;
  const int64_t each = block / bm, live = (routes / used + bm - 1) / bm;  // tiles of a block, with routes
  if (used >= kXcds || 2 * live <= each) run = (int)((run + each - 1) / each * each);
  return {bm, kCols, run};
}

}  // namespace

extern "C" int moe_mxfp4_quantize(const void* x, int dtype, int64_t rows, int K, int64_t row_stride,
                                  uint8_t* codes, uint8_t* scales, void* values, void* stream) {
  if (rows < 0 || K < 1 || K > 262144 || row_stride < K ||
      (dtype != MRS_DTYPE_F32 && dtype != MRS_DTYPE_BF16 && dtype != MRS_DTYPE_F16))
    return MRS_ERR_INVALID_ARG;
  if (rows == 0) return MRS_OK;
  if (!x || !codes || !scales) return MRS_ERR_NULL_POINTER;
  const int size = dtype == MRS_DTYPE_F32 ? 4 : 2;
  if (!aligned(x, size) || !aligned(codes, 4) || (values && !aligned(values, size))) return MRS_ERR_MISALIGNED;
  const int gpr = (K + 127) / 128 * 16;
  if (rows > (int64_t(1) << 38) / gpr) return MRS_ERR_OVERFLOW;
  const void* fn = dtype == MRS_DTYPE_F32    ? quant_kernel<MRS_DTYPE_F32>(values != nullptr)
                   : dtype == MRS_DTYPE_BF16 ? quant_kernel<MRS_DTYPE_BF16>(values != nullptr)
                                             : quant_kernel<MRS_DTYPE_F16>(values != nullptr);
  const int64_t most = kQLaunch / gpr;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = rows - r < most ? rows - r : most;
    QArgs a{static_cast<const char*>(x) + r * row_stride * size, codes + r * gpr * 4, scales + r * (gpr / 4),
            values ? static_cast<char*>(values) + r * K * size : nullptr, n, row_stride, n * gpr, K, gpr,
            (uint32_t)(((uint64_t(1) << 32) + gpr - 1) / gpr), ~uint64_t(0) / gpr + 1};
    const int64_t grid = (a.groups + kQThreads - 1) / kQThreads;
    void* params[] = {&a};
    if (hipLaunchKernel(fn, dim3((unsigned)grid), dim3(kQThreads), params, 0, reinterpret_cast<hipStream_t>(stream)) !=
        hipSuccess)
      return MRS_ERR_LAUNCH;
  }
  return MRS_OK;
}

extern "C" int moe_grouped_gemm_mxfp4(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                                      const uint8_t* w_scales, const int32_t* sorted_ids,
                                      const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k,
                                      int E, int K, int N, int block, int x_rows, int y_dtype, void* y,
                                      void* stream) {
  return moe_grouped_gemm_mxfp4_ex(x_codes, x_scales, w_codes, w_scales, sorted_ids, expert_of_block, num_post_pad, M,
                                   k, E, K, N, block, x_rows, y_dtype, y, stream, MRS_PRODUCT_BY_RULE);
}

extern "C" int moe_grouped_gemm_mxfp4_ex(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                                         const uint8_t* w_scales, const int32_t* sorted_ids,
                                         const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k,
                                         int E, int K, int N, int block, int x_rows, int y_dtype, void* y,
                                         void* stream, int kernel) {
  if (M < 0 || k < 1 || k > 64 || E < 1 || E > 4096 || K <= 0 || K > (1 << 22) || K % 128 != 0 || N < 1 || block < 16 ||
      block % 16 != 0 || (x_rows != MRS_X_TOKENS && x_rows != MRS_X_SORTED) ||
      (y_dtype != MRS_DTYPE_BF16 && y_dtype != MRS_DTYPE_F32) || kernel < MRS_PRODUCT_BY_RULE ||
      kernel > MRS_PRODUCT_TILE_128 || (kernel >= MRS_PRODUCT_TILE_16 && block % (16 << (kernel - MRS_PRODUCT_TILE_16))))
    return MRS_ERR_INVALID_ARG;
  const int64_t max_rows = moe_route_sort_max_rows(M, E, k, block);
  if (max_rows < 0) return MRS_ERR_OVERFLOW;
  const int64_t row_limit = max_rows / block * block;
  if (row_limit == 0) return MRS_OK;  // no token: nothing to write
  if (!x_codes || !x_scales || !w_codes || !w_scales || !sorted_ids || !expert_of_block || !num_post_pad || !y)
    return MRS_ERR_NULL_POINTER;
  if (!aligned(x_codes, 16) || !aligned(w_codes, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) ||
      !aligned(sorted_ids, 4) || !aligned(expert_of_block, 4) || !aligned(num_post_pad, 4) || !aligned(y, 4))
    return MRS_ERR_MISALIGNED;
  const int64_t routes = (int64_t)M * k, used = routes < E ? routes : E;
  const Shape shape = shape_of(routes, used, K, N, block, kernel);
  const int bm = shape.bm, bn = shape.bn;
  const int64_t nrt = row_limit / bm, ntn = ((int64_t)N + bn - 1) / bn;
  int64_t grid;
  if (bn < kCols) {  // whole rounds of pairs (padding block, column tile)
    const int64_t pairs = row_limit / block * ntn;
    grid = (pairs + kXcds * kPairs - 1) / (kXcds * kPairs) * (kXcds * kPairs) * (block / 16);
  } else {
    grid = (nrt + kXcds * shape.run - 1) / (kXcds * shape.run) * shape.run * kXcds * ntn;
  }
  if (grid * 256 > UINT32_MAX) return MRS_ERR_OVERFLOW;  // a launch has to have fewer than 2^32 threads
  PArgs a{x_codes, x_scales, w_codes, w_scales, sorted_ids, expert_of_block, num_post_pad, y,
          M, k, E, K, N, block, x_rows == MRS_X_SORTED, (int)row_limit, (int)nrt, (int)ntn, shape.run,
          (int64_t)E * N * K / 2 > 256 << 20};
  const void* fn = y_dtype == MRS_DTYPE_BF16 ? product_kernel<uint16_t>(bm, bn) : product_kernel<float>(bm, bn);
  void* params[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(256), params, 0,
                         reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? MRS_OK
             : MRS_ERR_LAUNCH;
}
