// 4-bit weights with group scales and the matrix-vector products of routed tokens,
// MI355X (gfx950, CDNA4, wave64).  Definitions: include/moe_int4.h.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "half.h"
#include "moe_int4.h"
#include "moe_route_sort.h"

namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------ quantisation
//
// A thread takes eight consecutive columns, so 4, 8 or 16 neighbouring lanes hold
// a group; its largest magnitude is the integer maximum of the bit patterns (which
// orders infinities and NaN above every number) over those lanes.

struct QArgs {
  const void* w;
  uint8_t* codes;
  uint16_t* scales;
  int64_t rows, stride;
  int K, gpr;          // gpr: eights of columns a row, Kp / 8
  uint32_t gpr_mul;    // ceil(2^32 / gpr): exact below 2^16, gpr <= 2^15
  uint64_t gpr_mul64;  // floor(2^64 / gpr) + 1: exact below 2^49
};

__device__ __forceinline__ uint32_t dpp_max(uint32_t v, uint32_t o) { return max(v, o); }

// Largest value of 4, 8 or 16 neighbouring lanes.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = dpp_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));  // quad_perm [1,0,3,2]
  v = dpp_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));  // quad_perm [2,3,0,1]
  if (LANES >= 8) v = dpp_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));  // half mirror
  if (LANES >= 16) v = dpp_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));  // mirror
  return v;
}

template <int DT>
__device__ __forceinline__ float value(const void* p, int64_t i) {
  if constexpr (DT == MRS_DTYPE_F32) return static_cast<const float*>(p)[i];
  else if constexpr (DT == MRS_DTYPE_BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  else return (float)static_cast<const _Float16*>(p)[i];
}

template <int DT, typename S, int GROUP>
__global__ __launch_bounds__(kThreads) void k_quantize(QArgs a) {
  const int64_t g0 = (int64_t)blockIdx.x * kThreads;
  const int64_t row0 = (int64_t)__umul64hi((uint64_t)g0, a.gpr_mul64);  // g0 / gpr
  const uint32_t in = (uint32_t)(g0 - row0 * a.gpr) + threadIdx.x;
  const uint32_t dr = __umulhi(in, a.gpr_mul);  // in / gpr
  const int64_t row = row0 + dr;
  const int g = (int)(in - dr * (uint32_t)a.gpr), c0 = g * 8;
  const bool live = row < a.rows;  // the same for the lanes of a group: gpr is a multiple of 16
  float v[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = live && c0 + i < a.K ? value<DT>(a.w, row * a.stride + c0 + i) : 0.0f;
    top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  }
  top = lanes_max<GROUP / 8>(top);
  const uint32_t packed = S::pack(__uint_as_float(top) / 7.0f, 0.0f);  // the scale, in the low half
  const float scale = S::lo(packed);
  const bool bad = !(scale < __uint_as_float(0x7F800000u));  // an infinity or a NaN
  uint32_t code = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = bad || scale == 0.0f ? 0.0f : fminf(fmaxf(rintf(v[i] / scale), -7.0f), 7.0f);
    code |= (uint32_t)((int)q + 8) << (4 * i);
  }
  if (!live) return;
  reinterpret_cast<uint32_t*>(a.codes)[row * a.gpr + g] = code;
  if (g % (GROUP / 8) == 0)
    a.scales[(row * a.gpr + g) / (GROUP / 8)] =
        bad ? (uint16_t)S::pack(__uint_as_float(0x7FC00000u), 0.0f) : (uint16_t)packed;
}

template <int DT, typename S>
const void* quant_kernel(int group) {
  return group == 32   ? reinterpret_cast<const void*>(k_quantize<DT, S, 32>)
         : group == 64 ? reinterpret_cast<const void*>(k_quantize<DT, S, 64>)
                       : reinterpret_cast<const void*>(k_quantize<DT, S, 128>);
}

template <typename S>
const void* quant_kernel(int dtype, int group) {
  return dtype == MRS_DTYPE_F32    ? quant_kernel<MRS_DTYPE_F32, S>(group)
         : dtype == MRS_DTYPE_BF16 ? quant_kernel<MRS_DTYPE_BF16, S>(group)
                                   : quant_kernel<MRS_DTYPE_F16, S>(group);
}

// A launch has to have fewer than 2^32 threads, and each takes one group of eight.
constexpr int64_t kQLaunch = int64_t(1) << 31;

// ---------------------------------------------------------- matrix-vector
//
// A lane takes chunks of 32 columns (16 bytes of codes): chunk q of the unit's
// contraction, the columns of one slot or (sum) those of a token's picks one after
// another.  L lanes share a row, so a wave works on 64 / L rows at once and R of
// such sets; it keeps its x values in registers and loads R sets of codes at a
// time.  A code c is made a 16-bit float by putting it into the top of the
// mantissa of 16.0: the value 16 + c costs one shift and one and-or for two codes,
// v_dot2 multiplies pairs into FP32, and 24 times the sum of x is taken off per
// chunk: sum x (16 + c) - 24 sum x = sum x (c - 8).  The partial sums are at most 55 sum |x|,
// whatever the codes, and are rounded 33 times (sum x, at 24, as often), so a chunk is off by up
// to 50 * 55 * 2^-24 scale sum |x|, also where its weights are all zero (codes 8).  Scale and pick
// weight enter once a chunk.  The low and high half of a dword's pair hold codes i and i + 4,
// so x is paired alike.
//
// Bound by the weights' bytes where there are many, by a chain of two round trips (the
// pick's id, then everything else) where there are few: one token of 896 experts,
// top-16, K 3584, N 768, gated: 23 MB in 8.3 us; 16 tokens 319 MB in 73 us, 4.4 TB/s;
// the second product and the sum of one token, 12 MB, 4.8 to 5.5 us.  64 tokens read shared
// experts again (872 MB once, 1.46 GB in all) and take 250 us, about half of it the
// 12 vector instructions for eight codes.

struct MArgs {
  const uint16_t* x;
  const uint8_t* codes;
  const uint16_t* scales;
  const int32_t* ids;
  const float* v;
  uint16_t* y;
  int M, k, E, K, N, per_slot;
  int chunks;   // of a row: Kp / 32
  int out;      // outputs of a slot: N, or N / 2 for gated results
  int tiles;    // workgroups of a slot (of a token for sums)
  uint32_t chunks_mul;  // ceil(2^32 / chunks)
};

template <typename H>
struct Magic;
template <>
struct Magic<BF16> {  // 7 bits of mantissa: 16 + c = 0x4180 | c << 3
  static constexpr uint32_t base = 0x41804180u, mask = 0x00780078u;
  static constexpr int at = 3;
  static constexpr uint32_t ones = 0x3F803F80u;
};
template <>
struct Magic<FP16> {  // 10 bits: 16 + c = 0x4C00 | c << 6
  static constexpr uint32_t base = 0x4C004C00u, mask = 0x03C003C0u;
  static constexpr int at = 6;
  static constexpr uint32_t ones = 0x3C003C00u;
};

// Codes i and i + 4 of a dword as 16 + c.  The constants are in registers (`mask`, `base`):
// as literals they would cost an instruction each.
template <typename H>
__device__ __forceinline__ uint32_t pair_of(uint32_t q, int i, uint32_t mask, uint32_t base) {
  const int up = Magic<H>::at - 4 * i;
  return ((up >= 0 ? q << up : q >> -up) & mask) | base;
}

// Sum over L neighbouring lanes, in the last of them.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v = add_dpp<0x111>(v);  // row_shr:1, 2, 4, 8
  v = add_dpp<0x112>(v);
  v = add_dpp<0x114>(v);
  if (L >= 16) v = add_dpp<0x118>(v);
  if (L >= 32) v = add_dpp<0x142>(v);  // the last lane of the row before
  if (L >= 64) v = add_dpp<0x143>(v);  // lane 31
  return v;
}

template <typename H, int MODE, int GROUP, int L, int R, int U>
__global__ __launch_bounds__(kThreads) void k_matvec(MArgs a) {
  constexpr int kSets = 64 / L;  // rows a wave works on at once
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
  const int q0 = lane % L, sub = lane / L;
  // gated: half of a wave's row sets are gates, the other half the columns they gate
  constexpr int kOut = MODE == MRS_INT4_GATED ? R / 2 : R;  // outputs of a lane's row sets
  const int n0 = (tile * (kThreads / 64) + wv) * kOut * kSets;
  if (n0 >= a.out) return;
  const int total = MODE == MRS_INT4_SUM ? a.k * a.chunks : a.chunks;
  int e = 0;
  if constexpr (MODE != MRS_INT4_SUM) {
    e = __builtin_amdgcn_readfirstlane(a.ids[unit]);
    if (e < 0 || e >= a.E) {
      for (int o = lane; o < kOut * kSets; o += 64)
        if (n0 + o < a.out) a.y[(int64_t)unit * a.out + n0 + o] = 0;
      return;
    }
  }
  uint32_t row[R];  // first chunk of a lane's rows, counted from the expert's
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int n = n0 + (r % kOut) * kSets + sub;
    row[r] = (uint32_t)(min(n, a.out - 1) + (r >= kOut ? a.out : 0)) * (uint32_t)a.chunks;
  }
  uint32_t mask = Magic<H>::mask, base = Magic<H>::base;
  asm volatile("" : "+v"(mask), "+v"(base));
  const int64_t matrix = (int64_t)a.N * a.chunks;  // chunks of an expert
  float acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = 0.0f;
  for (int b = 0; b < total; b += L * U) {
    u32x4 w[U][R], x[U][4];
    float sc[U][R], v[U];
    int left[U];  // values of x from a lane's chunk on, at most those of its row
    // everything that U chunks need is asked for before the first is used
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u * L >= total) continue;
      const int q = min(b + u * L + q0, total - 1);  // lanes past the last chunk repeat it and add nothing
      bool ok = b + u * L + q0 < total;
      int64_t slot = unit;
      int c = q, eu = e;
      v[u] = 1.0f;
      if constexpr (MODE == MRS_INT4_SUM) {
        const int j = (int)__umulhi((uint32_t)q, a.chunks_mul);  // q / chunks
        c = q - j * a.chunks;
        slot = (int64_t)unit * a.k + j;
        eu = a.ids[slot];
        v[u] = a.v[slot];
        ok = ok && eu >= 0 && eu < a.E;
        eu = eu >= 0 && eu < a.E ? eu : 0;
      }
      left[u] = ok ? a.K - c * 32 : 0;
      const int64_t xr = MODE == MRS_INT4_SUM ? (a.per_slot ? slot : unit) : (a.per_slot ? slot : slot / a.k);
      const uint16_t* xp = a.x + xr * a.K;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if (a.K >= 8) x[u][d] = *reinterpret_cast<const u32x4_any*>(xp + min(c * 32 + d * 8, a.K - 8));
        else x[u][d] = load_few(xp, ok && d == 0 && c == 0 ? a.K : 0);
      }
      const u32x4* codes = reinterpret_cast<const u32x4*>(a.codes) + eu * matrix;
      const uint16_t* scales = a.scales + eu * matrix / (GROUP / 32);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t at = row[r] + (uint32_t)c;
        w[u][r] = codes[at];
        sc[u][r] = H::lo(scales[at / (GROUP / 32)]);
        if (!ok) sc[u][r] = 0.0f;  // neither a scale's NaN nor a weight's
      }
      if (!ok) v[u] = 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u * L >= total) continue;
      if (a.K >= 8 && __ballot(left[u] < 32)) {  // the row ends in some lane's chunk: its last eight values, moved down
#pragma unroll
        for (int d = 0; d < 4; ++d) x[u][d] = drop(x[u][d], min(max(d * 8 + 8 - left[u], 0), 8));
      }
      uint32_t xs[16];
      float total_x = 0.0f;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const u32x4 p = x[u][d];
        // pairs (i, i + 4) of eight values: halves of dwords i / 2 and i / 2 + 2
        xs[4 * d] = __builtin_amdgcn_perm(p[2], p[0], 0x05040100u);
        xs[4 * d + 1] = __builtin_amdgcn_perm(p[2], p[0], 0x07060302u);
        xs[4 * d + 2] = __builtin_amdgcn_perm(p[3], p[1], 0x05040100u);
        xs[4 * d + 3] = __builtin_amdgcn_perm(p[3], p[1], 0x07060302u);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) total_x = H::dot2(xs[i], Magic<H>::ones, total_x);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float dot = -24.0f * total_x;
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) dot = H::dot2(pair_of<H>(w[u][r][d], i, mask, base), xs[4 * d + i], dot);
        acc[r] += MODE == MRS_INT4_SUM ? v[u] * (sc[u][r] * dot) : sc[u][r] * dot;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = lanes_sum<L>(acc[r]);
#pragma unroll
  for (int r = 0; r < kOut; ++r) {
    const int n = n0 + r * kSets + sub;
    float o = acc[r];
    if constexpr (MODE == MRS_INT4_GATED) o = o / (1.0f + __expf(-o)) * acc[r + kOut];
    if (q0 == L - 1 && n < a.out) a.y[(int64_t)unit * a.out + n] = (uint16_t)H::pack(o, 0.0f);
  }
}

struct MShape {
  int lanes, rows;  // lanes that share a row, row sets of a wave
};

template <typename H, int MODE, int GROUP, int R>
const void* matvec_kernel(int lanes) {
  constexpr int U = R == 4 ? 2 : 1;
  switch (lanes) {
    case 8: return reinterpret_cast<const void*>(k_matvec<H, MODE, GROUP, 8, R, U>);
    case 16: return reinterpret_cast<const void*>(k_matvec<H, MODE, GROUP, 16, R, U>);
    case 32: return reinterpret_cast<const void*>(k_matvec<H, MODE, GROUP, 32, R, U>);
    default: return reinterpret_cast<const void*>(k_matvec<H, MODE, GROUP, 64, R, U>);
  }
}

template <typename H, int MODE, int GROUP>
const void* matvec_kernel(MShape s) {
  return s.rows == 4 ? matvec_kernel<H, MODE, GROUP, 4>(s.lanes) : matvec_kernel<H, MODE, GROUP, 8>(s.lanes);
}

template <typename H, int MODE>
const void* matvec_kernel(int group, MShape s) {
  return group == 32 ? matvec_kernel<H, MODE, 32>(s)
         : group == 64 ? matvec_kernel<H, MODE, 64>(s)
                       : matvec_kernel<H, MODE, 128>(s);
}

template <typename H>
const void* matvec_kernel(int mode, int group, MShape s) {
  return mode == MRS_INT4_PLAIN   ? matvec_kernel<H, MRS_INT4_PLAIN>(group, s)
         : mode == MRS_INT4_GATED ? matvec_kernel<H, MRS_INT4_GATED>(group, s)
                                  : matvec_kernel<H, MRS_INT4_SUM>(group, s);
}

bool group_ok(int group) { return group == 32 || group == 64 || group == 128; }

}  // namespace

extern "C" int moe_int4_quantize(const void* w, int dtype, int64_t rows, int K, int64_t row_stride, int group,
                                 int scale_dtype, uint8_t* codes, void* scales, void* stream) {
  if (rows < 0 || K < 1 || K > 262144 || row_stride < K || !group_ok(group) ||
      (dtype != MRS_DTYPE_F32 && dtype != MRS_DTYPE_BF16 && dtype != MRS_DTYPE_F16) ||
      (scale_dtype != MRS_DTYPE_BF16 && scale_dtype != MRS_DTYPE_F16))
    return MRS_ERR_INVALID_ARG;
  if (rows == 0) return MRS_OK;
  if (!w || !codes || !scales) return MRS_ERR_NULL_POINTER;
  const int size = dtype == MRS_DTYPE_F32 ? 4 : 2;
  if (!aligned_to(w, size) || !aligned_to(codes, 4) || !aligned_to(scales, 2)) return MRS_ERR_MISALIGNED;
  const int gpr = (K + 127) / 128 * 16;
  if (rows > (int64_t(1) << 38) / gpr) return MRS_ERR_OVERFLOW;
  const void* fn = scale_dtype == MRS_DTYPE_BF16 ? quant_kernel<BF16>(dtype, group) : quant_kernel<FP16>(dtype, group);
  const int64_t most = kQLaunch / gpr;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = rows - r < most ? rows - r : most;
    QArgs a{static_cast<const char*>(w) + r * row_stride * size, codes + r * gpr * 4,
            static_cast<uint16_t*>(scales) + r * gpr * 8 / group, n, row_stride, K, gpr,
            (uint32_t)(((uint64_t(1) << 32) + gpr - 1) / gpr), ~uint64_t(0) / gpr + 1};
    void* params[] = {&a};
    if (hipLaunchKernel(fn, dim3((unsigned)((n * gpr + kThreads - 1) / kThreads)), dim3(kThreads), params, 0,
                        reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
      return MRS_ERR_LAUNCH;
  }
  return MRS_OK;
}

extern "C" int moe_int4_matvec(const void* x, int dtype, const uint8_t* codes, const void* scales, const int32_t* ids,
                               const float* weights, int M, int k, int E, int K, int N, int group, int per_slot,
                               int mode, void* y, void* stream) {
  if (M < 0 || k < 1 || k > 64 || E < 1 || E > 4096 || K < 1 || K > 262144 || N < 1 || N > 1 << 20 || !group_ok(group) ||
      (dtype != MRS_DTYPE_BF16 && dtype != MRS_DTYPE_F16) || mode < MRS_INT4_PLAIN || mode > MRS_INT4_SUM ||
      (mode == MRS_INT4_GATED && N % 2 != 0) ||
      (M > 0 && (weights != nullptr) != (mode == MRS_INT4_SUM)))  // an empty one has no address
    return MRS_ERR_INVALID_ARG;
  if ((int64_t)N * ((K + 127) / 128 * 4) > INT32_MAX / 16) return MRS_ERR_OVERFLOW;  // 32-bit offsets in a matrix
  if (M == 0) return MRS_OK;
  if (!x || !codes || !scales || !ids || !y) return MRS_ERR_NULL_POINTER;
  if (!aligned_to(x, 2) || !aligned_to(codes, 16) || !aligned_to(scales, 2) || !aligned_to(ids, 4) ||
      !aligned_to(weights, 4) || !aligned_to(y, 2))
    return MRS_ERR_MISALIGNED;
  MArgs a{static_cast<const uint16_t*>(x), codes, static_cast<const uint16_t*>(scales), ids, weights,
          static_cast<uint16_t*>(y), M, k, E, K, N, per_slot != 0, (K + 127) / 128 * 4,
          mode == MRS_INT4_GATED ? N / 2 : N, 0, 0};
  a.chunks_mul = (uint32_t)(((uint64_t(1) << 32) + a.chunks - 1) / a.chunks);
  const int total = mode == MRS_INT4_SUM ? k * a.chunks : a.chunks;
  const int64_t units = mode == MRS_INT4_SUM ? M : (int64_t)M * k;
  // Eight row sets share the work on x, four with two chunks at once come to more waves
  // with more in flight: the rule's border is where the times cross (us, 8 / 4; workgroups
  // of 8: one token of 896 experts, top-16, K 3584, N 768 gated, 384: 9.8 / 8.3; 4 tokens,
  // 1536: 19.0 / 20.7; 64 tokens, 24576: 248 / 278; the sum of K 384, N 3584, 112: 7.9 / 6.2;
  // 33 tokens, top-4 of 64, K 1001, N 515, 1188: 11.0 / 11.6; 40 tokens, top-4 of 16, K 500,
  // N 600, 800: 8.2 / 7.5).
  MShape shape{total >= 64 ? 64 : total >= 32 ? 32 : total >= 16 ? 16 : 8, 8};
  auto tiles = [&] {
    const int outs = (mode == MRS_INT4_GATED ? shape.rows / 2 : shape.rows) * (64 / shape.lanes) * (kThreads / 64);
    return (a.out + outs - 1) / outs;
  };
  if (units * tiles() < 1024) shape.rows = 4;
  a.tiles = tiles();
  const int64_t grid = units * a.tiles;
  if (grid * kThreads > UINT32_MAX) return MRS_ERR_OVERFLOW;
  const void* fn = dtype == MRS_DTYPE_BF16 ? matvec_kernel<BF16>(mode, group, shape) : matvec_kernel<FP16>(mode, group, shape);
  void* params[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(kThreads), params, 0, reinterpret_cast<hipStream_t>(stream)) ==
                 hipSuccess
             ? MRS_OK
             : MRS_ERR_LAUNCH;
}
