// Balance loss, per-expert counts and the router's gradient, MI355X (gfx950,
// CDNA4, wave64).  Definitions and argument contracts: include/moe_balance.h.
//
// Both directions read each row of logits once: a wave takes a row, its lanes
// hold the row's scores in registers, a wave-wide sum gives the row's total.
// Forward: the waves of a workgroup walk a chunk of tokens, each adding its
// rows' shares into registers; the workgroup's column sums and its LDS
// histogram of the ids go to the workspace as one piece per (chunk, sequence),
// and a second kernel adds the pieces up in their order.  Backward: the row's
// counts-weighted mean comes from the same registers, and the picks' gradient
// joins in FP32 before the one rounding.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_balance.h"
#include "moe_route_sort.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;
constexpr float kLog2e = 1.44269504088896340736f;
// A row total below this is renormalised from shifted logits: above it a score
// that FP32 flushes to zero (below 2^-126) is under 2^-66 of the total.
constexpr float kTiny = 0x1p-60f;

struct BArgs {
  const void* logits;
  const int32_t* ids;
  const int32_t* off;   // null: one sequence
  const uint8_t* mask;  // null: every token
  int M, E, k, B, chunk, chunks;
  float coef;
  // forward
  float* loss;
  int32_t* counts;
  int32_t* tokens;
  float* shares;
  float* ws_share;      // [pieces, E]
  int32_t* ws_count;    // [pieces, E]
  int32_t* ws_n;        // [pieces]
  double* ws_loss;      // [B * tiles]
  uint32_t* ws_ticket;
  // backward
  const float* grad_w;
  const float* grad_loss;
  void* out;
};

__device__ __forceinline__ float lane_value(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float old, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, ROWS, 0xF, false));
}

// Sum over the wave, the same in every lane: row shifts by 1, 2, 4, 8, then the
// rows' last lanes passed on, total in lane 63.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x111, 0xF>(0.0f, v);
  v += dpp<0x112, 0xF>(0.0f, v);
  v += dpp<0x114, 0xF>(0.0f, v);
  v += dpp<0x118, 0xF>(0.0f, v);
  v += dpp<0x142, 0xA>(0.0f, v);
  v += dpp<0x143, 0xC>(0.0f, v);
  return lane_value(v, 63);
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, 64));
  return v;
}

__device__ __forceinline__ float fast_rcp(float v) { return __builtin_amdgcn_rcpf(v); }
__device__ __forceinline__ float fast_exp(float v) { return __builtin_amdgcn_exp2f(v * kLog2e); }

// s = sigmoid(x) and s (1 - s), both from u = exp(-|x|) <= 1, so neither
// overflows nor cancels; NaN passes through.
__device__ __forceinline__ float sigmoid(float x, float& slope) {
  const float u = fast_exp(-__builtin_fabsf(x));
  const float r = fast_rcp(1.0f + u), ur = u * r;
  slope = ur * r;
  return x >= 0.0f ? r : (x != x ? x : ur);
}
__device__ __forceinline__ float sigmoid(float x) { return fast_rcp(1.0f + fast_exp(-x)); }

template <int DT>
struct Row;
template <>
struct Row<MRS_DTYPE_F32> {
  typedef float T;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Row<MRS_DTYPE_BF16> {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t put(float v) {  // to nearest even; NaN stays NaN
    const uint32_t u = __float_as_uint(v);
    return v != v ? (uint16_t)0x7FC0u : (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
  }
};

// VEC consecutive columns (one load) at column (i * 64 + lane) * VEC; columns
// past E read as -infinity, whose score is zero.
template <int DT, int VEC, int NI>
__device__ __forceinline__ void load_row(const typename Row<DT>::T* row, int E, int lane, float (&x)[NI][VEC]) {
  typedef typename Row<DT>::T T;
  struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
  };
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = (i * 64 + lane) * VEC;
    const Pack p = *reinterpret_cast<const Pack*>(row + (c < E ? c : 0));
#pragma unroll
    for (int v = 0; v < VEC; ++v) x[i][v] = c < E ? Row<DT>::get(p.v[v]) : -__builtin_inff();
  }
}

// Offset of sequence b, inside [0, M].
__device__ __forceinline__ int offset_of(const BArgs& a, int b) {
  if (!a.off) return b == 0 ? 0 : a.M;
  return min(max(a.off[b], 0), a.M);
}

// The sequence that holds token t: the last b < B with off[b] <= t.
__device__ __forceinline__ int sequence_of(const BArgs& a, int t) {
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offset_of(a, mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// p of a row in place of its logits: s / sum s, or exp(x - max) / sum where the
// total underflows (there sigmoid(x) and exp(x) agree far past FP32).
template <int VEC, int NI>
__device__ __forceinline__ void shares_of_row(float (&x)[NI][VEC]) {
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int v = 0; v < VEC; ++v) m = fmaxf(m, x[i][v]);
  m = wave_max(m);
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      x[i][v] = m > -__builtin_inff() ? fast_exp(x[i][v] - m) : 0.0f;
      total += x[i][v];
    }
  total = wave_sum(total);
  const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int v = 0; v < VEC; ++v) x[i][v] *= inv;
}

// Piece c + b holds chunk c's part of sequence b: along the tokens every next
// (chunk, sequence) pair raises c or b, so no two pairs share a piece.
template <int DT, int VEC, int NI>
__global__ __launch_bounds__(kThreads) void k_balance_part(BArgs a) {
  typedef typename Row<DT>::T T;
  extern __shared__ char lds[];
  float* share = reinterpret_cast<float*>(lds);                  // [E]
  int32_t* hist = reinterpret_cast<int32_t*>(lds) + a.E;         // [E]
  __shared__ int live_tokens;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = blockIdx.x;
  if (c == 0 && tid == 0) *a.ws_ticket = 0u;
  const int t_end = min(a.M, (c + 1) * a.chunk);
  int t0 = c * a.chunk;
  for (int b = sequence_of(a, t0); b < a.B && t0 < t_end; ++b) {
    const int t1 = b == a.B - 1 ? t_end : min(offset_of(a, b + 1), t_end);
    if (t1 <= t0) continue;
    for (int e = tid; e < a.E; e += kThreads) {
      share[e] = 0.0f;
      hist[e] = 0;
    }
    if (tid == 0) live_tokens = 0;
    __syncthreads();
    float acc[NI][VEC];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) acc[i][v] = 0.0f;
    int n = 0;
    for (int t = t0 + wv; t < t1; t += kWaves) {
      if (a.mask && !a.mask[t]) continue;
      ++n;
      if (lane < a.k) {
        const int id = a.ids[(size_t)t * a.k + lane];
        if (id >= 0 && id < a.E) atomicAdd(&hist[id], 1);
      }
      float x[NI][VEC];
      const T* row = static_cast<const T*>(a.logits) + (size_t)t * a.E;
      load_row<DT, VEC, NI>(row, a.E, lane, x);
      float s[NI][VEC], total = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          s[i][v] = sigmoid(x[i][v]);
          total += s[i][v];
        }
      total = wave_sum(total);
      if (total < kTiny) {
        shares_of_row<VEC, NI>(x);
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < VEC; ++v) acc[i][v] += x[i][v];
      } else {
        const float inv = 1.0f / total;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < VEC; ++v) acc[i][v] = fmaf(s[i][v], inv, acc[i][v]);
      }
    }
    if (lane == 0) atomicAdd(&live_tokens, n);
    for (int w = 0; w < kWaves; ++w) {  // in wave order
      if (wv == w)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < VEC; ++v) {
            const int e = (i * 64 + lane) * VEC + v;
            if (e < a.E) share[e] += acc[i][v];
          }
      __syncthreads();
    }
    const size_t piece = (size_t)(c + b);
    for (int e = tid; e < a.E; e += kThreads) {
      a.ws_share[piece * a.E + e] = share[e];
      a.ws_count[piece * a.E + e] = hist[e];
    }
    if (tid == 0) a.ws_n[piece] = live_tokens;
    __syncthreads();
    t0 = t1;
  }
}

constexpr int kTile = 64;  // experts a workgroup of the second kernel adds up

__global__ __launch_bounds__(kThreads) void k_balance_sum(BArgs a) {
  __shared__ double sh[kWaves][kTile];
  __shared__ int ct[kWaves][kTile], nn[kWaves];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int tiles = gridDim.x, b = blockIdx.y;
  const int e = blockIdx.x * kTile + lane;
  const int t0 = offset_of(a, b), t1 = b == a.B - 1 ? a.M : offset_of(a, b + 1);
  int first = 0, end = 0;
  if (t1 > t0) {
    first = t0 / a.chunk + b;
    end = (t1 - 1) / a.chunk + b + 1;
  }
  double s = 0.0;
  int count = 0, n = 0;
  for (int p = first + wv; p < end; p += kWaves) {
    if (e < a.E) {
      s += (double)a.ws_share[(size_t)p * a.E + e];
      count += a.ws_count[(size_t)p * a.E + e];
    }
    n += a.ws_n[p];
  }
  sh[wv][lane] = s;
  ct[wv][lane] = count;
  if (lane == 0) nn[wv] = n;
  __syncthreads();
  if (wv == 0) {
    n = nn[0] + nn[1] + nn[2] + nn[3];
    s = ((sh[0][lane] + sh[1][lane]) + sh[2][lane]) + sh[3][lane];
    count = ct[0][lane] + ct[1][lane] + ct[2][lane] + ct[3][lane];
    const double share = n > 0 ? s / n : 0.0;
    if (e < a.E) {
      a.counts[(size_t)b * a.E + e] = count;
      a.shares[(size_t)b * a.E + e] = (float)share;
    }
    double part = e < a.E && n > 0 ? (double)count * share / n : 0.0;
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) part += __shfl_xor(part, m, 64);
    if (lane == 0) {
      a.ws_loss[(size_t)b * tiles + blockIdx.x] = part;
      if (blockIdx.x == 0) a.tokens[b] = n;
    }
  }
  // the workgroup that finishes last adds the tiles up in their order
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    last = atomicAdd(a.ws_ticket, 1u) == (uint32_t)tiles * (uint32_t)a.B - 1u;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  double total = 0.0;
  int filled = 0;
  for (int i = tid; i < tiles * a.B; i += kThreads) total += __hip_atomic_load(&a.ws_loss[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = tid; i < a.B; i += kThreads)
    filled += __hip_atomic_load(&a.tokens[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 0;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    total += __shfl_xor(total, m, 64);
    filled += __shfl_xor(filled, m, 64);
  }
  if (lane == 0) {
    sh[wv][0] = total;
    nn[wv] = filled;
  }
  __syncthreads();
  if (tid == 0) {
    filled = nn[0] + nn[1] + nn[2] + nn[3];
    total = ((sh[0][0] + sh[1][0]) + sh[2][0]) + sh[3][0];
    a.tokens[a.B] = filled;
    a.loss[0] = filled > 0 ? (float)((double)a.coef * total * a.E / ((double)a.k * filled)) : 0.0f;
  }
}

// No token: zeros, one workgroup.
__global__ __launch_bounds__(kThreads) void k_balance_none(BArgs a) {
  for (size_t i = threadIdx.x; i < (size_t)a.B * a.E; i += kThreads) {
    a.counts[i] = 0;
    a.shares[i] = 0.0f;
  }
  for (int i = threadIdx.x; i <= a.B; i += kThreads) a.tokens[i] = 0;
  if (threadIdx.x == 0) a.loss[0] = 0.0f;
}

// d/dx of the balance loss of row t: g_b s' / S * (count[b,e] - sum_e' count[b,e'] p[e']),
// g_b = grad_loss coef E / (k n_b^2 B'); of the picks' weights:
// w_j (1 - s_j) (grad_w_j - sum_i grad_w_i w_i), added through a row of LDS.
template <int DT, int VEC, int NI>
__global__ __launch_bounds__(kThreads) void k_router_backward(BArgs a) {
  typedef typename Row<DT>::T T;
  extern __shared__ char lds[];
  float* cnt = reinterpret_cast<float*>(lds);                                     // [E]
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  float* extra = reinterpret_cast<float*>(lds) + (size_t)a.E * (1 + wv);          // [E] of this wave
  const int c = blockIdx.x;
  const int t_end = min(a.M, (c + 1) * a.chunk);
  int t0 = c * a.chunk;
  for (int e = lane; e < a.E; e += 64) extra[e] = 0.0f;
  const float gl = a.grad_loss ? *a.grad_loss : 1.0f;
  const int filled = a.counts ? a.tokens[a.B] : 0;
  for (int b = sequence_of(a, t0); b < a.B && t0 < t_end; ++b) {
    const int t1 = b == a.B - 1 ? t_end : min(offset_of(a, b + 1), t_end);
    if (t1 <= t0) continue;
    __syncthreads();
    if (a.counts)
      for (int e = tid; e < a.E; e += kThreads) cnt[e] = (float)a.counts[(size_t)b * a.E + e];
    const int n = a.counts ? a.tokens[b] : 0;
    const float g = n > 0 && filled > 0
                        ? (float)((double)gl * a.coef * a.E / ((double)a.k * n * (double)n * filled))
                        : 0.0f;
    __syncthreads();
    for (int t = t0 + wv; t < t1; t += kWaves) {
      T* dst = static_cast<T*>(a.out) + (size_t)t * a.E;
      struct alignas(sizeof(T) * VEC) Pack {
        T v[VEC];
      };
      if (a.mask && !a.mask[t]) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int e = (i * 64 + lane) * VEC;
          if (e < a.E) *reinterpret_cast<Pack*>(dst + e) = Pack{};
        }
        continue;
      }
      const T* row = static_cast<const T*>(a.logits) + (size_t)t * a.E;
      int id = -1;
      float gw = 0.0f, xk = -__builtin_inff();
      if (a.grad_w && lane < a.k) {
        id = a.ids[(size_t)t * a.k + lane];
        gw = a.grad_w[(size_t)t * a.k + lane];
        if (id < 0 || id >= a.E) {
          id = -1;
          gw = 0.0f;
        } else {
          xk = Row<DT>::get(row[id]);
        }
      }
      float d[NI][VEC], cv[NI][VEC], dot = 0.0f, scale = 0.0f;
      if (a.counts) {
        float x[NI][VEC], s[NI][VEC], total = 0.0f;
        load_row<DT, VEC, NI>(row, a.E, lane, x);
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < VEC; ++v) {
            s[i][v] = sigmoid(x[i][v], d[i][v]);
            total += s[i][v];
          }
        total = wave_sum(total);
        if (total < kTiny) {
          shares_of_row<VEC, NI>(x);
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int v = 0; v < VEC; ++v) s[i][v] = d[i][v] = x[i][v];
          scale = 1.0f;
        } else {
          scale = 1.0f / total;
        }
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < VEC; ++v) {
            const int e = (i * 64 + lane) * VEC + v;
            cv[i][v] = e < a.E ? cnt[e] : 0.0f;
            dot = fmaf(cv[i][v], s[i][v], dot);
          }
        dot = wave_sum(dot) * scale;
      }
      if (a.grad_w) {
        // scores of the picks relative to exp(min(max x, 0)), so they never all underflow
        const float m = fminf(wave_max(xk), 0.0f);
        float w = 0.0f, rest = 0.0f;
        if (id >= 0 && m > -__builtin_inff()) {
          const float u = fast_exp(-__builtin_fabsf(xk));
          const float r = fast_rcp(1.0f + u);
          w = xk > 0.0f ? r : (xk != xk ? xk : fast_exp(xk - m) * r);  // s / exp(m)
          rest = xk > 0.0f ? u * r : r;                                // 1 - s
        }
        const float sum = wave_sum(w);
        w = sum > 0.0f || sum != sum ? w / sum : 0.0f;
        const float mean = wave_sum(gw * w);
        if (id >= 0) atomicAdd(&extra[id], w * rest * (gw - mean));
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // other lanes read it below
      }
      const float f = g * scale;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int e = (i * 64 + lane) * VEC;
        if (e < a.E) {
          Pack o;
#pragma unroll
          for (int v = 0; v < VEC; ++v) {
            const float add = a.grad_w ? extra[e + v] : 0.0f;
            o.v[v] = Row<DT>::put(a.counts ? fmaf((cv[i][v] - dot) * f, d[i][v], add) : add);
          }
          *reinterpret_cast<Pack*>(dst + e) = o;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (id >= 0) extra[id] = 0.0f;
    }
    t0 = t1;
  }
}

constexpr int kMaxChunks = 1024;

int choose_chunk(int M) {
  int c = (M + kMaxChunks - 1) / kMaxChunks;
  c = (c + kWaves - 1) / kWaves * kWaves;
  return c < 2 * kWaves ? 2 * kWaves : c;
}

size_t align16(size_t v) { return (v + 15) & ~size_t(15); }

struct Plan {
  int chunk, chunks, tiles;
  size_t share, count, n, loss, ticket, total;
};

Plan plan_of(int M, int E, int B) {
  Plan p{};
  p.chunk = choose_chunk(M);
  p.chunks = (M + p.chunk - 1) / p.chunk;
  p.tiles = (E + kTile - 1) / kTile;
  const size_t pieces = (size_t)p.chunks + B;
  p.share = 0;
  p.count = p.share + align16(pieces * E * 4);
  p.n = p.count + align16(pieces * E * 4);
  p.loss = p.n + align16(pieces * 4);
  p.ticket = p.loss + align16((size_t)B * p.tiles * 8);
  p.total = p.ticket + 16;
  return p;
}

bool valid_sizes(int M, int E, int k, int B) {
  return M >= 0 && E >= 1 && E <= 4096 && k >= 1 && k <= 64 && B >= 1 && B <= 65535;
}

enum { kPart, kBack };

template <int WHAT, int DT, int VEC, int NI>
const void* one() {
  if constexpr (WHAT == kPart) return reinterpret_cast<const void*>(k_balance_part<DT, VEC, NI>);
  else return reinterpret_cast<const void*>(k_router_backward<DT, VEC, NI>);
}

template <int WHAT, int DT>
const void* pick(int E, bool even) {
  if (even) {
    const int ni = (E + 127) / 128;
    if (ni <= 1) return one<WHAT, DT, 2, 1>();
    if (ni <= 2) return one<WHAT, DT, 2, 2>();
    if (ni <= 3) return one<WHAT, DT, 2, 3>();
    if (ni <= 4) return one<WHAT, DT, 2, 4>();
    if (ni <= 6) return one<WHAT, DT, 2, 6>();
    if (ni <= 7) return one<WHAT, DT, 2, 7>();
    if (ni <= 8) return one<WHAT, DT, 2, 8>();
    if (ni <= 12) return one<WHAT, DT, 2, 12>();
    if (ni <= 16) return one<WHAT, DT, 2, 16>();
    if (ni <= 24) return one<WHAT, DT, 2, 24>();
    return one<WHAT, DT, 2, 32>();
  }
  const int ni = (E + 63) / 64;
  if (ni <= 2) return one<WHAT, DT, 1, 2>();
  if (ni <= 8) return one<WHAT, DT, 1, 8>();
  if (ni <= 24) return one<WHAT, DT, 1, 24>();
  return one<WHAT, DT, 1, 64>();
}

template <int WHAT>
const void* kernel_of(int dtype, int E, bool even) {
  return dtype == MRS_DTYPE_F32 ? pick<WHAT, MRS_DTYPE_F32>(E, even) : pick<WHAT, MRS_DTYPE_BF16>(E, even);
}

int launch(const void* fn, dim3 grid, size_t lds, BArgs& a, void* stream) {
  void* params[] = {&a};
  return hipLaunchKernel(fn, grid, dim3(kThreads), params, lds, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? MRS_OK
             : MRS_ERR_LAUNCH;
}

}  // namespace

extern "C" size_t moe_balance_workspace_bytes(int M, int E, int k, int B) {
  if (!valid_sizes(M, E, k, B)) return (size_t)-1;
  return plan_of(M, E, B).total;
}

extern "C" int moe_balance_loss(const void* logits, int logits_dtype, const int32_t* ids, const int32_t* seq_offsets,
                                const uint8_t* mask, int M, int E, int k, int B, float coef, float* loss,
                                int32_t* counts, int32_t* tokens, float* shares, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!valid_sizes(M, E, k, B) || (!seq_offsets && B != 1) ||
      (logits_dtype != MRS_DTYPE_F32 && logits_dtype != MRS_DTYPE_BF16))
    return MRS_ERR_INVALID_ARG;
  if (!loss || !counts || !tokens || !shares) return MRS_ERR_NULL_POINTER;
  if (!aligned(loss, 4) || !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(shares, 4))
    return MRS_ERR_MISALIGNED;
  const Plan p = plan_of(M, E, B);
  BArgs a{};
  a.logits = logits;
  a.ids = ids;
  a.off = seq_offsets;
  a.mask = mask;
  a.M = M;
  a.E = E;
  a.k = k;
  a.B = B;
  a.chunk = p.chunk;
  a.chunks = p.chunks;
  a.coef = coef;
  a.loss = loss;
  a.counts = counts;
  a.tokens = tokens;
  a.shares = shares;
  if (M == 0) return launch(reinterpret_cast<const void*>(k_balance_none), dim3(1), 0, a, stream);
  if (!logits || !ids) return MRS_ERR_NULL_POINTER;
  const int size = logits_dtype == MRS_DTYPE_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(ids, 4) || !aligned(seq_offsets, 4)) return MRS_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < p.total) return MRS_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return MRS_ERR_MISALIGNED;
  char* ws = static_cast<char*>(workspace);
  a.ws_share = reinterpret_cast<float*>(ws + p.share);
  a.ws_count = reinterpret_cast<int32_t*>(ws + p.count);
  a.ws_n = reinterpret_cast<int32_t*>(ws + p.n);
  a.ws_loss = reinterpret_cast<double*>(ws + p.loss);
  a.ws_ticket = reinterpret_cast<uint32_t*>(ws + p.ticket);
  const bool even = E % 2 == 0 && aligned(logits, 2 * size);
  int rc = launch(kernel_of<kPart>(logits_dtype, E, even), dim3(p.chunks), (size_t)E * 8, a, stream);
  if (rc == MRS_OK) rc = launch(reinterpret_cast<const void*>(k_balance_sum), dim3(p.tiles, B), 0, a, stream);
  return rc;
}

extern "C" int moe_router_backward(const void* logits, int logits_dtype, const int32_t* ids, const float* grad_w,
                                   const int32_t* counts, const int32_t* tokens, const float* grad_loss,
                                   const int32_t* seq_offsets, const uint8_t* mask, int M, int E, int k, int B,
                                   float coef, void* grad_logits, void* stream) {
  if (!valid_sizes(M, E, k, B) || (!seq_offsets && B != 1) ||
      (logits_dtype != MRS_DTYPE_F32 && logits_dtype != MRS_DTYPE_BF16))
    return MRS_ERR_INVALID_ARG;
  if (M == 0) return MRS_OK;
  if (!logits || !ids || !grad_logits || (counts && !tokens)) return MRS_ERR_NULL_POINTER;
  const int size = logits_dtype == MRS_DTYPE_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(grad_logits, size) || !aligned(ids, 4) || !aligned(grad_w, 4) ||
      !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(grad_loss, 4) || !aligned(seq_offsets, 4))
    return MRS_ERR_MISALIGNED;
  BArgs a{};
  a.logits = logits;
  a.ids = ids;
  a.off = seq_offsets;
  a.mask = mask;
  a.M = M;
  a.E = E;
  a.k = k;
  a.B = B;
  a.chunk = choose_chunk(M);
  a.chunks = (M + a.chunk - 1) / a.chunk;
  a.coef = coef;
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.grad_w = grad_w;
  a.grad_loss = grad_loss;
  a.out = grad_logits;
  const bool even = E % 2 == 0 && aligned(logits, 2 * size) && aligned(grad_logits, 2 * size);
  return launch(kernel_of<kBack>(logits_dtype, E, even), dim3(a.chunks), (size_t)E * 4 * (1 + kWaves), a, stream);
}
