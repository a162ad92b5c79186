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
  uint32_t gpr_mul;              // ceil(2^32 / gpr)
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

// VEC: 16-byte accesses (rows of x aligned, K a multiple of 8).  Every lane of
// a quad belongs to the same row (gpr is a multiple of 16) and all of them run.
template <int DT, bool VEC, bool VALUES>
__global__ __launch_bounds__(kQThreads) void k_quantize(QArgs a) {
  typedef Elem<DT> El;
  typedef typename El::T T;
  const int64_t g0 = (int64_t)blockIdx.x * kQThreads;
  const int64_t row0 = g0 / a.gpr;
  const uint32_t in = (uint32_t)(g0 - row0 * a.gpr) + threadIdx.x;
  const uint32_t dr = __umulhi(in, a.gpr_mul);  // in / gpr
  const int64_t row = row0 + dr;
  const int g = (int)(in - dr * (uint32_t)a.gpr), c0 = g * 8;
  const bool live = row < a.rows;
  const T* src = static_cast<const T*>(a.x) + row * a.stride + c0;
  T raw[8];
  if (VEC) {
    if (live && c0 < a.K) {
#pragma unroll
      for (int i = 0; i < (int)(8 * sizeof(T) / 16); ++i)
        reinterpret_cast<u32x4*>(raw)[i] = reinterpret_cast<const u32x4*>(src)[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[i] = T(0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = live && c0 + i < a.K ? src[i] : T(0);
  }
  float v[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = El::get(raw[i]);
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
    T o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      o[i] = El::put(bad ? __uint_as_float(0x7FC00000u) : ldexpf(d[i / 2][i % 2], (int)X - 127));
    if (VEC) {
      if (c0 < a.K)
#pragma unroll
        for (int i = 0; i < (int)(8 * sizeof(T) / 16); ++i)
          reinterpret_cast<u32x4*>(dst)[i] = reinterpret_cast<u32x4*>(o)[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + i < a.K) dst[i] = o[i];
    }
  }
}

template <int DT>
const void* quant_kernel(bool vec, bool values) {
  if (vec)
    return values ? reinterpret_cast<const void*>(k_quantize<DT, true, true>)
                  : reinterpret_cast<const void*>(k_quantize<DT, true, false>);
  return values ? reinterpret_cast<const void*>(k_quantize<DT, false, true>)
                : reinterpret_cast<const void*>(k_quantize<DT, false, false>);
}

// --------------------------------------------------------- grouped product

struct PArgs {
  const uint8_t *xc, *xs, *wc, *ws;
  const int32_t *sid, *eob, *npp;
  void* y;
  int M, k, E, K, N, block, sorted;
  int row_limit;  // rows the metadata can hold: (max_rows / block) * block
  int nrt, ntn;   // row tiles, column tiles
};

// Workgroup h goes to XCD h mod 8; runs of kRunRows consecutive row tiles go to
// the XCDs in turn and, inside a run, the row tiles of one column tile come one
// after another, so the row tiles of an expert read its weights from one L2.
constexpr int kXcds = 8;
constexpr int kRunRows = 8;
__device__ __forceinline__ bool tile_of(int h, int ntn, int nrt, int& rt, int& ct) {
  const int x = h % kXcds, j = h / kXcds;
  const int m = j / (kRunRows * ntn), c = (j / kRunRows) % ntn, r = j % kRunRows;
  rt = (m * kXcds + x) * kRunRows + r;
  ct = c;
  return rt < nrt;
}

__device__ __forceinline__ void put_y(float* y, float v) { *y = v; }
// FP32 to BF16, round to nearest even; NaN stays NaN.
__device__ __forceinline__ void put_y(uint16_t* y, float v) {
  const uint32_t u = __float_as_uint(v);
  const uint32_t r = u + 0x7FFFu + ((u >> 16) & 1u);
  *y = v != v ? (uint16_t)0x7FC0u : (uint16_t)(r >> 16);
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
// LDS but the partial sums.  Padding rows load nothing.
template <typename Y, int FN, int U>
__global__ __launch_bounds__(256) void k_product_rows(PArgs a) {
  __shared__ f32x4 part[4][FN][64];
  int rt, ct;
  if (!tile_of((int)blockIdx.x, a.ntn, a.nrt, rt, ct)) return;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  const int r0 = rt * 16, n0 = ct * 16 * FN;
  const int npp = min(*a.npp, a.row_limit);
  const int e = a.eob[r0 / a.block];
  const int s = a.sid[r0 + r16];
  if (r0 >= npp || e < 0 || e >= a.E) return;
  const bool ok = s >= 0 && s < a.M * a.k;
  const uint32_t rows = (uint32_t)__ballot(ok) & 0xFFFFu;
  f32x4 acc[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) acc[j] = f32x4{};
  if (rows) {
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
    const int steps = a.K / 128;
    for (int t0 = wv; t0 < steps; t0 += 4 * U) {
      u32x4 xq[U], wq[U][FN];
      int xe[U], we[U][FN];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = min(t0 + 4 * u, steps - 1);
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
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t0 + 4 * u < steps)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                frag(xq[u]), frag(wq[u][j]), acc[j], 4, 4, 0, (int)((uint32_t)xe[u] >> (8 * q)), 0,
                (int)((uint32_t)we[u][j] >> (8 * q)));
    }
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
// l mod 32).  Steps of 256 columns: the x rows are shared by the waves and
// staged through two LDS buffers (rows of 128 bytes, 16-byte chunks XOR-swizzled
// so that the 32 rows of an operand read hit distinct banks); each wave's
// weights are its own and go from memory to its registers, the next step's
// while the present one is multiplied.
template <int CH>
__device__ __forceinline__ int swz(int r, int c) {
  return r * CH + (c ^ (r & 7) ^ ((r >> 3) & 1));
}

struct __attribute__((packed, aligned(4))) Scale8 {
  uint32_t lo, hi;
};

template <typename Y, int BM, int FM>
__device__ __forceinline__ void tile_body(const PArgs& a, int r0, int n0, int e, u32x4 (*xl)[BM * 8],
                                          Scale8 (*sl)[BM]) {
  constexpr int XP = BM * 8 / 256;  // x chunks a thread stages in a step
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int lr = lane & 31, lh = lane >> 5;
  const int routes = a.M * a.k;
  const size_t kb = (size_t)a.K / 2, ks = (size_t)a.K / 32;
  const int steps = (a.K + 255) / 256;
  const bool half = a.K % 256 != 0;  // the last step has 128 columns

  const uint8_t* xsrc[XP];
  bool xok[XP];
#pragma unroll
  for (int p = 0; p < XP; ++p) {
    const int r = (tid + p * 256) / 8, c = tid % 8;
    const int s = a.sid[r0 + r];
    xok[p] = s >= 0 && s < routes;
    const size_t row = xok[p] ? (size_t)(a.sorted ? r0 + r : s / a.k) : 0;
    xsrc[p] = a.xc + row * kb + c * 16;
  }
  const uint8_t* ssrc = a.xs;
  bool sok = false;
  if (tid < BM) {
    const int s = a.sid[r0 + tid];
    sok = s >= 0 && s < routes;
    const size_t row = sok ? (size_t)(a.sorted ? r0 + tid : s / a.k) : 0;
    ssrc = a.xs + row * ks;
  }
  const uint8_t *wc[2], *ws[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const size_t n = (size_t)e * a.N + min(n0 + wv * 64 + j * 32 + lr, a.N - 1);
    wc[j] = a.wc + n * kb + lh * 16;
    ws[j] = a.ws + n * ks;
  }

  u32x4 xr[XP];
  Scale8 sr;
  u32x4 wq[2][4];
  uint32_t we[2][2];
  // a step's second half past the end of K is not read: zero codes and scales
  auto load_x = [&](int t) {
    const bool full = !(half && t == steps - 1);
#pragma unroll
    for (int p = 0; p < XP; ++p) {
      xr[p] = u32x4{0u, 0u, 0u, 0u};
      if (xok[p] && (full || tid % 8 < 4)) xr[p] = *reinterpret_cast<const u32x4*>(xsrc[p] + (size_t)t * 128);
    }
    sr.lo = sr.hi = 0u;
    if (sok) {
      sr.lo = *reinterpret_cast<const uint32_t*>(ssrc + t * 8);
      if (full) sr.hi = *reinterpret_cast<const uint32_t*>(ssrc + t * 8 + 4);
    }
  };
  auto store_x = [&](int buf) {
#pragma unroll
    for (int p = 0; p < XP; ++p) xl[buf][swz<8>((tid + p * 256) / 8, tid % 8)] = xr[p];
    if (tid < BM) sl[buf][tid] = sr;
  };
  auto load_w = [&](int t, u32x4 (&q)[2][4], uint32_t (&s)[2][2]) {
    const bool full = !(half && t == steps - 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[j][i] = u32x4{0u, 0u, 0u, 0u};
        if (i < 2 || full) q[j][i] = *reinterpret_cast<const u32x4*>(wc[j] + (size_t)t * 128 + i * 32);
      }
      s[j][0] = *reinterpret_cast<const uint32_t*>(ws[j] + t * 8);
      s[j][1] = full ? *reinterpret_cast<const uint32_t*>(ws[j] + t * 8 + 4) : 0u;
    }
  };

  f32x16 acc[FM][2];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};

  load_x(0);
  load_w(0, wq, we);
  store_x(0);
  __syncthreads();
  for (int t = 0; t < steps; ++t) {
    const int cur = t & 1;
    u32x4 wn[2][4];
    uint32_t wne[2][2];
    const bool more = t + 1 < steps;
    if (more) {
      load_x(t + 1);
      load_w(t + 1, wn, wne);
    }
    // scale of columns 64 g + 32 lh ..: byte 2 (g mod 2) of the word g / 2 shifted by 8 lh
    uint32_t xe[FM][2];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const Scale8 v = sl[cur][i * 32 + lr];
      xe[i][0] = v.lo >> (8 * lh);
      xe[i][1] = v.hi >> (8 * lh);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      i32x8 xf[FM], wf[2];
#pragma unroll
      for (int i = 0; i < FM; ++i) xf[i] = frag(xl[cur][swz<8>(i * 32 + lr, 2 * g + lh)]);
#pragma unroll
      for (int j = 0; j < 2; ++j) wf[j] = frag(wq[j][g]);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int sx = (int)xe[i][g / 2], sw = (int)(we[j][g / 2] >> (8 * lh));
          if (g % 2 == 0)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xf[i], wf[j], acc[i][j], 4, 4, 0, sx, 0, sw);
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xf[i], wf[j], acc[i][j], 4, 4, 2, sx, 2, sw);
        }
    }
    if (more) {
      store_x(cur ^ 1);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) wq[j][i] = wn[j][i];
        we[j][0] = wne[j][0];
        we[j][1] = wne[j][1];
      }
    }
    __syncthreads();
  }

  // result register v of lane l: row 8 (v / 4) + 4 (l / 32) + v mod 4, column l mod 32
#pragma unroll
  for (int i = 0; i < BM / 32; ++i) {
    const int sr32 = a.sid[r0 + i * 32 + lr];
    const uint32_t rows = (uint32_t)__ballot(sr32 >= 0 && sr32 < routes);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = n0 + wv * 64 + j * 32 + lr;
      if (n < a.N)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int r = 8 * (v / 4) + 4 * lh + v % 4;
          float o = 0.0f;
          if (i < FM) o = (rows >> r) & 1u ? acc[i < FM ? i : 0][j][v] : 0.0f;
          put_y(static_cast<Y*>(a.y) + (size_t)(r0 + i * 32 + r) * a.N + n, o);
        }
    }
  }
}

template <typename Y, int BM>
__global__ __launch_bounds__(256) void k_product_tile(PArgs a) {
  __shared__ u32x4 xl[2][BM * 8];
  __shared__ Scale8 sl[2][BM];
  int rt, ct;
  if (!tile_of((int)blockIdx.x, a.ntn, a.nrt, rt, ct)) return;
  const int r0 = rt * BM;
  const int npp = min(*a.npp, a.row_limit);
  if (r0 + BM > npp) return;  // npp is a multiple of block and BM divides block
  const int e = a.eob[r0 / a.block];
  if (e < 0 || e >= a.E) return;
  // a segment's routes come first: the last 32 rows that hold one bound the work
  int live = 0;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < BM / 32; ++i) {
    const int s = a.sid[r0 + i * 32 + (lane & 31)];
    if (__ballot(s >= 0 && s < a.M * a.k)) live = i + 1;
  }
  live = __builtin_amdgcn_readfirstlane(live);
  if constexpr (BM == 128) {
    if (live == 4) return tile_body<Y, BM, 4>(a, r0, ct * 256, e, xl, sl);
    if (live == 3) return tile_body<Y, BM, 3>(a, r0, ct * 256, e, xl, sl);
  }
  if constexpr (BM >= 64) {
    if (live == 2) return tile_body<Y, BM, 2>(a, r0, ct * 256, e, xl, sl);
  }
  return tile_body<Y, BM, 1>(a, r0, ct * 256, e, xl, sl);
}

template <typename Y>
const void* product_kernel(int bm) {
  switch (bm) {
    case 128: return reinterpret_cast<const void*>(k_product_tile<Y, 128>);
    case 64: return reinterpret_cast<const void*>(k_product_tile<Y, 64>);
    case 32: return reinterpret_cast<const void*>(k_product_tile<Y, 32>);
    default: return reinterpret_cast<const void*>(k_product_rows<Y, 1, 4>);
  }
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
  QArgs a{x, codes, scales, values, rows, row_stride, rows * gpr, K, gpr,
          (uint32_t)(((uint64_t(1) << 32) + gpr - 1) / gpr)};
  const bool vec = aligned(x, 16) && (!values || aligned(values, 16)) && K % 8 == 0 && row_stride * size % 16 == 0;
  const int64_t grid = (a.groups + kQThreads - 1) / kQThreads;
  const void* fn = dtype == MRS_DTYPE_F32    ? quant_kernel<MRS_DTYPE_F32>(vec, values != nullptr)
                   : dtype == MRS_DTYPE_BF16 ? quant_kernel<MRS_DTYPE_BF16>(vec, values != nullptr)
                                             : quant_kernel<MRS_DTYPE_F16>(vec, values != nullptr);
  void* params[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(kQThreads), params, 0,
                         reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? MRS_OK
             : MRS_ERR_LAUNCH;
}

extern "C" int moe_grouped_gemm_mxfp4(const uint8_t* x_codes, const uint8_t* x_scales, const uint8_t* w_codes,
                                      const uint8_t* w_scales, const int32_t* sorted_ids,
                                      const int32_t* expert_of_block, const int32_t* num_post_pad, int M, int k,
                                      int E, int K, int N, int block, int x_rows, int y_dtype, void* y,
                                      void* stream) {
  if (M < 0 || k < 1 || k > 64 || E < 1 || E > 4096 || K <= 0 || K % 128 != 0 || N < 1 || block < 16 ||
      block % 16 != 0 || (x_rows != MRS_X_TOKENS && x_rows != MRS_X_SORTED) ||
      (y_dtype != MRS_DTYPE_BF16 && y_dtype != MRS_DTYPE_F32))
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
  int bm = 16;
  if (block % 32 == 0 && routes > 16 * used) {
    bm = block % 128 == 0 && routes > 64 * used ? 128 : (block % 64 == 0 && routes > 32 * used ? 64 : 32);
  }
  const int bn = bm == 16 ? 16 : 256;
  const int64_t nrt = row_limit / bm, ntn = ((int64_t)N + bn - 1) / bn;
  const int64_t runs = (nrt + kXcds * kRunRows - 1) / (kXcds * kRunRows) * kRunRows;
  if (runs * kXcds * ntn > INT32_MAX) return MRS_ERR_OVERFLOW;
  PArgs a{x_codes, x_scales, w_codes, w_scales, sorted_ids, expert_of_block, num_post_pad, y,
          M, k, E, K, N, block, x_rows == MRS_X_SORTED, (int)row_limit, (int)nrt, (int)ntn};
  const void* fn = y_dtype == MRS_DTYPE_BF16 ? product_kernel<uint16_t>(bm) : product_kernel<float>(bm);
  void* params[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)(runs * kXcds * ntn)), dim3(256), params, 0,
                         reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? MRS_OK
             : MRS_ERR_LAUNCH;
}
