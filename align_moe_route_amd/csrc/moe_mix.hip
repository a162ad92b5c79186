// The gated activation and the mix of the experts' outputs, forward and backward,
// MI355X (gfx950, CDNA4, wave64).  Definitions: include/moe_experts.h.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "half.h"
#include "moe_experts.h"
#include "moe_route_sort.h"

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + __expf(-x)); }

template <typename H>
struct Eight {
  float v[8];
  __device__ __forceinline__ void get(u32x4 q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = H::lo(q[i]);
      v[2 * i + 1] = H::hi(q[i]);
    }
  }
  __device__ __forceinline__ u32x4 put() const {
    return u32x4{H::pack(v[0], v[1]), H::pack(v[2], v[3]), H::pack(v[4], v[5]), H::pack(v[6], v[7])};
  }
};

// ------------------------------------------------------------- activation
//
// A thread takes eight columns of a row; `gpr` groups of eight a row, the row of a
// thread by a host-made multiplier in place of a division.  Rows need no more
// alignment than their elements.  Bound by memory: 188416 rows of I 384, of which 85 % count,
// 62 us, 5.9 TB/s (a part of it in the cache in front of the memory); the gradient of 40000
// rows of I 1001 in FP16 71 us, 5.1 TB/s.

struct SArgs {
  const uint16_t *a, *dh;
  const int32_t* npp;
  uint16_t* out;
  int64_t rows;
  int I, gpr;
  uint32_t gpr_mul;    // ceil(2^32 / gpr): exact below 2^17 + 2^8
  uint64_t gpr_mul64;  // floor(2^64 / gpr) + 1: exact below 2^49
};

template <typename H, bool GRAD>
__global__ __launch_bounds__(kThreads) void k_swiglu(SArgs s) {
  const int64_t g0 = (int64_t)blockIdx.x * kThreads;
  const int64_t row0 = s.gpr == 1 ? g0 : (int64_t)__umul64hi((uint64_t)g0, s.gpr_mul64);  // g0 / gpr
  const uint32_t in = (uint32_t)(g0 - row0 * s.gpr) + threadIdx.x;
  const uint32_t dr = s.gpr == 1 ? in : __umulhi(in, s.gpr_mul);  // in / gpr
  const int64_t row = row0 + dr;
  int64_t rows = s.rows;
  if (s.npp) rows = min(rows, (int64_t)*s.npp);
  if (row >= rows) return;
  const int c = (int)(in - dr * (uint32_t)s.gpr) * 8, n = s.I - c;
  const uint16_t* a = s.a + row * 2 * s.I + c;
  Eight<H> g, u, o;
  g.get(load8(a, n));
  u.get(load8(a + s.I, n));
  if constexpr (GRAD) {
    Eight<H> d, p;
    d.get(load8(s.dh + row * s.I + c, n));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sg = sigmoid(g.v[i]);
      o.v[i] = d.v[i] * u.v[i] * sg * (1.0f + g.v[i] * (1.0f - sg));
      p.v[i] = d.v[i] * g.v[i] * sg;
    }
    uint16_t* da = s.out + row * 2 * s.I + c;
    store8(da, o.put(), n);
    store8(da + s.I, p.put(), n);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = g.v[i] * sigmoid(g.v[i]) * u.v[i];
    store8(s.out + row * s.I + c, o.put(), n);
  }
}

// ------------------------------------------------------------------ slots

__global__ __launch_bounds__(kThreads) void k_fill_rows(int32_t* rows, int n) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i < n) rows[i] = -1;
}

__global__ __launch_bounds__(kThreads) void k_slot_rows(const int32_t* sid, const int32_t* npp, int capacity,
                                                        int32_t* rows, int n) {
  const int r = blockIdx.x * kThreads + threadIdx.x;
  if (r >= min(*npp, capacity)) return;
  const int s = sid[r];
  if (s >= 0 && s < n) rows[s] = r;
}

// Few slots: one workgroup and one launch, through LDS, up to where it takes as long as the
// two (us, one launch / two; 4 slots 1.8 / 3.4, 1024 slots in 14464 rows 2.7 / 3.5, 8192 in
// 12224 3.6 / 3.9, 16384 in 20416 5.5 / 3.9), which also cost the host another launch.
constexpr int kSlotThreads = 1024, kFewSlots = 8192, kFewRows = 16384;
__global__ __launch_bounds__(kSlotThreads) void k_slot_rows_few(const int32_t* sid, const int32_t* npp, int capacity,
                                                                int32_t* rows, int n) {
  __shared__ int32_t at[kFewSlots];
  const int end = min(*npp, capacity);
  for (int i = threadIdx.x; i < n; i += kSlotThreads) at[i] = -1;
  __syncthreads();
  for (int r = threadIdx.x; r < end; r += kSlotThreads) {
    const int s = sid[r];
    if (s >= 0 && s < n) at[s] = r;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kSlotThreads) rows[i] = at[i];
}

// -------------------------------------------------------------------- mix
//
// A wave takes 512 columns of a token, eight a lane, and its picks in turn, eight
// loads in flight; rows and weights are the same for every lane.  Bound by memory: 8192
// tokens, top-16, N 3584 180 us, 5.5 TB/s.

struct CArgs {
  const uint16_t* y;
  const int32_t *rows, *sid, *npp;
  const float* v;
  const uint16_t* dout;
  void* out;
  float* dv;
  int64_t capacity;
  int M, k, N, segs;
};

constexpr int kDeep = 8;

template <typename H, bool F32>
__global__ __launch_bounds__(kThreads) void k_combine(CArgs a) {
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (int)(unit / a.segs), c = (int)(unit % a.segs) * 512 + (threadIdx.x & 63) * 8;
  if (t >= a.M) return;
  const int n = a.N - c;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
  const int64_t s0 = (int64_t)t * a.k;
  for (int j = 0; j < a.k; j += kDeep) {
    u32x4 q[kDeep];
    float v[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      q[i] = u32x4{0u, 0u, 0u, 0u};
      v[i] = 0.0f;
      if (j + i < a.k) {
        const int64_t r = a.rows ? a.rows[s0 + j + i] : s0 + j + i;
        if (r >= 0 && r < a.capacity) {
          v[i] = a.v ? a.v[s0 + j + i] : 1.0f;
          q[i] = load8(a.y + r * a.N + c, n);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      Eight<H> e;
      e.get(q[i]);
#pragma unroll
      for (int x = 0; x < 8; ++x) sum[x] += v[i] * e.v[x];
    }
  }
  if constexpr (F32) {
    float* o = static_cast<float*>(a.out) + (int64_t)t * a.N + c;
#pragma unroll
    for (int x = 0; x < 8; ++x)
      if (x < n) o[x] = sum[x];
  } else {
    Eight<H> e;
#pragma unroll
    for (int x = 0; x < 8; ++x) e.v[x] = sum[x];
    store8(static_cast<uint16_t*>(a.out) + (int64_t)t * a.N + c, e.put(), n);
  }
}

// Sum over the 64 lanes of a wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// A wave takes a slot; the workgroups past the slots' zero the padding rows, 64 a
// wave.  A token's row of dout is read once for each of its picks, by waves that run
// together.  Bound by memory: 8192 tokens, top-8, N 3584, with the weights' gradient 220 us,
// 4.7 TB/s.
template <typename H, bool DOT>
__global__ __launch_bounds__(kThreads) void k_combine_backward(CArgs a, int slot_blocks) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint16_t* dy = static_cast<uint16_t*>(a.out);
  const int64_t routes = (int64_t)a.M * a.k;
  if ((int)blockIdx.x >= slot_blocks) {
    const int64_t r0 = ((int64_t)((int)blockIdx.x - slot_blocks) * (kThreads / 64) + wv) * 64;
    const int64_t end = min((int64_t)*a.npp, a.capacity);
    bool pad = false;
    if (r0 + lane < end) {
      const int s = a.sid[r0 + lane];
      pad = s < 0 || s >= routes;
    }
    for (uint64_t m = __ballot(pad); m; m &= m - 1) {
      uint16_t* p = dy + (r0 + __builtin_ctzll(m)) * a.N;
      for (int c = lane * 8; c < a.N; c += 512) store8(p + c, u32x4{0u, 0u, 0u, 0u}, a.N - c);
    }
    return;
  }
  const int64_t s = (int64_t)blockIdx.x * (kThreads / 64) + wv;
  if (s >= routes) return;
  const int64_t r = a.rows[s];
  const bool ok = r >= 0 && r < a.capacity;
  if (!ok) {
    if (DOT && lane == 0) a.dv[s] = 0.0f;
    return;
  }
  const float v = a.v ? a.v[s] : 1.0f;
  const uint16_t* d = a.dout + s / a.k * a.N;
  float dot = 0.0f;
  for (int c = lane * 8; c < a.N; c += 512) {
    Eight<H> e, y;
    e.get(load8(d + c, a.N - c));
    if constexpr (DOT) {
      y.get(load8(a.y + r * a.N + c, a.N - c));
#pragma unroll
      for (int x = 0; x < 8; ++x) dot += e.v[x] * y.v[x];
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) e.v[x] *= v;
    store8(dy + r * a.N + c, e.put(), a.N - c);
  }
  if constexpr (DOT) {
    dot = wave_sum(dot);
    if (lane == 0) a.dv[s] = dot;
  }
}

bool half_dtype(int dtype) { return dtype == MRS_DTYPE_BF16 || dtype == MRS_DTYPE_F16; }

constexpr int kMaxCols = 1 << 20;

int launch(const void* fn, int64_t grid, void** params, void* stream, int threads = kThreads) {
  return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(threads), params, 0, reinterpret_cast<hipStream_t>(stream)) ==
                 hipSuccess
             ? MRS_OK
             : MRS_ERR_LAUNCH;
}

int swiglu(const void* a, const void* dh, bool grad, int dtype, const int32_t* npp, int64_t rows, int I, void* out,
           void* stream) {
  if (rows < 0 || rows > INT32_MAX || I < 1 || I > 262144 || !half_dtype(dtype)) return MRS_ERR_INVALID_ARG;
  if (rows == 0) return MRS_OK;
  if (!a || !out || (grad && !dh)) return MRS_ERR_NULL_POINTER;
  if (!aligned_to(a, 2) || !aligned_to(out, 2) || !aligned_to(dh, 2) || !aligned_to(npp, 4)) return MRS_ERR_MISALIGNED;
  const int gpr = (I + 7) / 8;
  if (rows > (int64_t(1) << 31) / gpr) return MRS_ERR_OVERFLOW;  // a launch has to have fewer than 2^32 threads
  const void* fn = dtype == MRS_DTYPE_BF16 ? (grad ? reinterpret_cast<const void*>(k_swiglu<BF16, true>)
                                                   : reinterpret_cast<const void*>(k_swiglu<BF16, false>))
                                           : (grad ? reinterpret_cast<const void*>(k_swiglu<FP16, true>)
                                                   : reinterpret_cast<const void*>(k_swiglu<FP16, false>));
  SArgs s{static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(dh), npp, static_cast<uint16_t*>(out), rows, I, gpr,
          (uint32_t)(((uint64_t(1) << 32) + gpr - 1) / gpr), ~uint64_t(0) / gpr + 1};
  void* params[] = {&s};
  return launch(fn, (rows * gpr + kThreads - 1) / kThreads, params, stream);
}

}  // namespace

extern "C" int moe_swiglu(const void* a, int dtype, const int32_t* num_post_pad, int64_t rows, int I, void* h,
                          void* stream) {
  return swiglu(a, nullptr, false, dtype, num_post_pad, rows, I, h, stream);
}

extern "C" int moe_swiglu_backward(const void* a, const void* dh, int dtype, const int32_t* num_post_pad, int64_t rows,
                                   int I, void* da, void* stream) {
  return swiglu(a, dh, true, dtype, num_post_pad, rows, I, da, stream);
}

extern "C" int moe_slot_rows(const int32_t* sorted_ids, const int32_t* num_post_pad, int64_t capacity, int M, int k,
                             int32_t* rows, void* stream) {
  if (capacity < 0 || M < 0 || k < 1 || k > 64) return MRS_ERR_INVALID_ARG;
  if (capacity > INT32_MAX - kThreads || (int64_t)M * k > INT32_MAX - kThreads) return MRS_ERR_OVERFLOW;
  if (M == 0) return MRS_OK;
  if (!sorted_ids || !num_post_pad || !rows) return MRS_ERR_NULL_POINTER;
  if (!aligned_to(sorted_ids, 4) || !aligned_to(num_post_pad, 4) || !aligned_to(rows, 4)) return MRS_ERR_MISALIGNED;
  int n = M * k, cap = (int)capacity;
  if (n <= kFewSlots && cap <= kFewRows) {
    void* params[] = {&sorted_ids, &num_post_pad, &cap, &rows, &n};
    return launch(reinterpret_cast<const void*>(k_slot_rows_few), 1, params, stream, kSlotThreads);
  }
  void* fill[] = {&rows, &n};
  const int rc = launch(reinterpret_cast<const void*>(k_fill_rows), (n + kThreads - 1) / kThreads, fill, stream);
  if (rc != MRS_OK || cap == 0) return rc;
  void* params[] = {&sorted_ids, &num_post_pad, &cap, &rows, &n};
  return launch(reinterpret_cast<const void*>(k_slot_rows), (cap + kThreads - 1) / kThreads, params, stream);
}

extern "C" int moe_combine(const void* y, int dtype, const int32_t* rows, const float* weights, int64_t capacity, int M,
                           int k, int N, int out_dtype, void* out, void* stream) {
  if (capacity < 0 || M < 0 || k < 1 || k > 64 || N < 1 || N > kMaxCols || !half_dtype(dtype) ||
      (out_dtype != dtype && out_dtype != MRS_DTYPE_F32))
    return MRS_ERR_INVALID_ARG;
  if ((int64_t)M * k > INT32_MAX || capacity > INT32_MAX) return MRS_ERR_OVERFLOW;
  if (M == 0) return MRS_OK;
  if ((!y && capacity > 0) || !out) return MRS_ERR_NULL_POINTER;
  if (!aligned_to(y, 2) || !aligned_to(rows, 4) || !aligned_to(weights, 4) ||
      !aligned_to(out, out_dtype == MRS_DTYPE_F32 ? 4 : 2))
    return MRS_ERR_MISALIGNED;
  CArgs a{};
  a.y = static_cast<const uint16_t*>(y), a.rows = rows, a.v = weights, a.out = out, a.capacity = capacity;
  a.M = M, a.k = k, a.N = N, a.segs = (N + 511) / 512;
  const int64_t grid = ((int64_t)M * a.segs + kThreads / 64 - 1) / (kThreads / 64);
  if (grid * kThreads > UINT32_MAX) return MRS_ERR_OVERFLOW;
  const bool f32 = out_dtype == MRS_DTYPE_F32;
  const void* fn = dtype == MRS_DTYPE_BF16 ? (f32 ? reinterpret_cast<const void*>(k_combine<BF16, true>)
                                                  : reinterpret_cast<const void*>(k_combine<BF16, false>))
                                           : (f32 ? reinterpret_cast<const void*>(k_combine<FP16, true>)
                                                  : reinterpret_cast<const void*>(k_combine<FP16, false>));
  void* params[] = {&a};
  return launch(fn, grid, params, stream);
}

extern "C" int moe_combine_backward(const void* dout, const void* y, int dtype, const int32_t* rows,
                                    const int32_t* sorted_ids, const int32_t* num_post_pad, const float* weights,
                                    int64_t capacity, int M, int k, int N, void* dy, float* dweights, void* stream) {
  if (capacity < 0 || M < 0 || k < 1 || k > 64 || N < 1 || N > kMaxCols || !half_dtype(dtype) ||
      (M > 0 && !y != !dweights))  // an empty dweights has no address
    return MRS_ERR_INVALID_ARG;
  if ((int64_t)M * k > INT32_MAX || capacity > INT32_MAX) return MRS_ERR_OVERFLOW;
  if (M == 0) return MRS_OK;
  if (!dout || !rows || !sorted_ids || !num_post_pad || !dy) return MRS_ERR_NULL_POINTER;
  if (!aligned_to(dout, 2) || !aligned_to(y, 2) || !aligned_to(rows, 4) || !aligned_to(sorted_ids, 4) ||
      !aligned_to(num_post_pad, 4) || !aligned_to(weights, 4) || !aligned_to(dy, 2) || !aligned_to(dweights, 4))
    return MRS_ERR_MISALIGNED;
  CArgs a{};
  a.y = static_cast<const uint16_t*>(y), a.rows = rows, a.sid = sorted_ids, a.npp = num_post_pad, a.v = weights;
  a.dout = static_cast<const uint16_t*>(dout), a.out = dy, a.dv = dweights, a.capacity = capacity;
  a.M = M, a.k = k, a.N = N;
  int slot_blocks = (int)(((int64_t)M * k + kThreads / 64 - 1) / (kThreads / 64));
  const int64_t grid = slot_blocks + (capacity + kThreads - 1) / kThreads;
  if (grid * kThreads > UINT32_MAX) return MRS_ERR_OVERFLOW;
  const void* fn = dtype == MRS_DTYPE_BF16 ? (y ? reinterpret_cast<const void*>(k_combine_backward<BF16, true>)
                                                : reinterpret_cast<const void*>(k_combine_backward<BF16, false>))
                                           : (y ? reinterpret_cast<const void*>(k_combine_backward<FP16, true>)
                                                : reinterpret_cast<const void*>(k_combine_backward<FP16, false>));
  void* params[] = {&a, &slot_blocks};
  return launch(fn, grid, params, stream);
}
