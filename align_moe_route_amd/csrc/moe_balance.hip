// Balance loss, per-expert counts and the router's gradient, MI355X (gfx950,
// CDNA4, wave64).  Definitions and argument contracts: include/moe_balance.h.
//
// Both directions read each row of logits once: sixteen lanes (up to 256
// experts), a wave (up to 1024) or four waves take a row, up to sixteen columns of
// it to a thread, the next rows on their way meanwhile; a thread keeps its columns
// (their running shares, or their counts) in registers throughout.
// Forward: a workgroup walks a chunk of tokens; its column sums and its LDS
// histogram of the ids go to the workspace as one piece per (chunk, sequence),
// and a second kernel adds the pieces up in their order (one workgroup alone
// finishes a small batch itself).  Backward: the row's counts-weighted mean comes
// from the same pass, and the picks' gradient joins in FP32 before the one
// rounding.
//
// Bound by the logits' bytes where there are many (a 2 GiB copy moves 4.9 TB/s).
// With the same inputs call after call, which the 256 MB cache keeps in part:
// forward 16384 x 4096 FP32, 37 sequences, in 60 us (276 MB, 4.6 TB/s; the pieces
// add 37 MB and two small launches 11 us), 65536 x 512 FP32 in 30 us; backward 99
// and 46 us (541 and 273 MB, 5.5 and 5.9 TB/s).  With other inputs each time the
// first of them takes 68 us forward and 112 backward (4.0 and 4.8 TB/s).
// 8192 x 896 BF16 takes 15.5 us forward, 8 of them the second launch's chain of
// round trips, and 11 us backward (30 MB; 6 us of arithmetic, the rest latency);
// 131072 x 128 BF16 20 and 22 us.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_balance.h"
#include "moe_route_sort.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr float kLog2e = 1.44269504088896340736f;
// A row total below this is renormalised from shifted logits: above it a score
// that FP32 flushes to zero (below 2^-126) is under 2^-66 of the total.
constexpr float kTiny = 0x1p-60f;

struct BArgs {
  const void* logits;
  const int32_t* ids;
  const int32_t* off;   // null: one sequence
  const uint8_t* mask;  // null: every token
  int M, E, k, B, chunk;
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

// Reductions over segments of S lanes, the same bits in each lane of a segment.
template <int S>
__device__ __forceinline__ float seg_sum(float v) {
  if constexpr (S == 64) return wave_sum(v);
  v += dpp<0x128, 0xF>(0.0f, v);  // rows of 16 lanes rotated by 8, 4, 2, 1
  v += dpp<0x124, 0xF>(0.0f, v);
  v += dpp<0x122, 0xF>(0.0f, v);
  return v + dpp<0x121, 0xF>(0.0f, v);
}
template <int S>
__device__ __forceinline__ float seg_max(float v) {
  if constexpr (S == 64) return wave_max(v);
  v = fmaxf(v, dpp<0x128, 0xF>(0.0f, v));
  v = fmaxf(v, dpp<0x124, 0xF>(0.0f, v));
  v = fmaxf(v, dpp<0x122, 0xF>(0.0f, v));
  return fmaxf(v, dpp<0x121, 0xF>(0.0f, v));
}

__device__ __forceinline__ float fast_rcp(float v) { return __builtin_amdgcn_rcpf(v); }
__device__ __forceinline__ float fast_exp(float v) { return __builtin_amdgcn_exp2f(v * kLog2e); }

// s = sigmoid(x) and s (1 - s), both from u = exp(-|x|) <= 1, so neither
// overflows nor cancels; NaN passes through.
__device__ __forceinline__ float sigmoid(float x, float& slope) {
  const float u = fast_exp(-__builtin_fabsf(x));
  const float r = fast_rcp(1.0f + u), ur = u * r;
  slope = ur * r;
  return x >= 0.0f ? r : ur;
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
  // to nearest even, NaN stays NaN (v_cvt_pk_bf16_f32)
  static __device__ __forceinline__ uint16_t put(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};

// G threads of a workgroup share a row; a thread has NI times four columns, at
// (i G + its place in the group) * 4.
constexpr int kThreads = 256;  // of a workgroup, but for the forward pass (part_threads)

// Four columns from c of a row of E, as stored; columns past E read as -infinity,
// whose score is zero.  Rows need no more alignment than their elements.
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(4)));
template <int DT>
union Four;
template <>
union Four<MRS_DTYPE_F32> {
  typedef u32x4_any Wide;
  float v[4];
  u32x4_any w;
};
template <>
union Four<MRS_DTYPE_BF16> {
  typedef u32x2_any Wide;
  uint16_t v[4];
  u32x2_any w;
};
// `inner`: of a thread's column groups all but the last lie inside the row.
template <int DT>
__device__ __forceinline__ Four<DT> load4(const typename Row<DT>::T* row, int c, int E, bool inner) {
  Four<DT> q;
  if (inner || c + 4 <= E) {
    q.w = *reinterpret_cast<const typename Four<DT>::Wide*>(row + c);
    return q;
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) q.v[v] = c + v < E ? row[c + v] : Row<DT>::put(-__builtin_inff());
  return q;
}
// Past the L2, where the logits to come are worth more than the gradient that no
// thread reads again (us: 8192 x 896 BF16 13.4 -> 11.8, 16384 x 4096 FP32 120 -> 109,
// 65536 x 512 FP32 64 -> 48).
template <int DT>
__device__ __forceinline__ void store4(typename Row<DT>::T* row, int c, int E, bool inner, const float (&x)[4]) {
  if (inner || c + 4 <= E) {
    Four<DT> q;
#pragma unroll
    for (int v = 0; v < 4; ++v) q.v[v] = Row<DT>::put(x[v]);
    __builtin_nontemporal_store(q.w, reinterpret_cast<typename Four<DT>::Wide*>(row + c));
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (c + v < E) row[c + v] = Row<DT>::put(x[v]);
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

// Sum or maximum over a group, the same bits in each of its threads.  `box` holds
// a word for each of the group's waves; every thread of a group calls it together.
template <int G>
__device__ __forceinline__ float group_sum(float v, float* box) {
  v = seg_sum<G < 64 ? G : 64>(v);
  if constexpr (G > 64) {
    if ((threadIdx.x & 63) == 0) box[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < G / 64; ++w) v += box[w];
    __syncthreads();
  }
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v, float* box) {
  v = seg_max<G < 64 ? G : 64>(v);
  if constexpr (G > 64) {
    if ((threadIdx.x & 63) == 0) box[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < G / 64; ++w) v = fmaxf(v, box[w]);
    __syncthreads();
  }
  return v;
}

// out[r] = sum over the W waves of box[w * R + r], the same bits in every lane:
// the W R words spread over the lanes, lane l with row l mod R, and a butterfly.
template <int W, int R>
__device__ __forceinline__ void sum_waves(const float* box, float (&out)[R]) {
  constexpr int V = W * R, L = V < 64 ? V : 64;
  const int lane = threadIdx.x & 63;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < V; i += 64) v += box[i + lane % L];
#pragma unroll
  for (int m = R; m < L; m *= 2) v += __shfl_xor(v, m, 64);
#pragma unroll
  for (int r = 0; r < R; ++r) out[r] = lane_value(v, r);
}

// Shares of a row whose total underflows: exp(x - max) / sum (there sigmoid(x)
// and exp(x) agree far past FP32); zero where every logit is -infinity.
template <int DT, int G, int NI>
__device__ __forceinline__ void far_shares(const typename Row<DT>::T* row, int c0, int E, float* box, float (&p)[NI][4]) {
  float m = -__builtin_inff(), total = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const Four<DT> q = load4<DT>(row, c0 + i * G * 4, E, i < NI - 1);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      p[i][v] = Row<DT>::get(q.v[v]);
      m = fmaxf(m, p[i][v]);
    }
  }
  m = group_max<G>(m, box);
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      p[i][v] = m > -__builtin_inff() ? fast_exp(p[i][v] - m) : 0.0f;
      total += p[i][v];
    }
  total = group_sum<G>(total, box);
  const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) p[i][v] *= inv;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

__device__ __forceinline__ float loss_of(const BArgs& a, double total, int filled) {
  return filled > 0 ? (float)((double)a.coef * total * a.E / ((double)a.k * filled)) : 0.0f;
}

constexpr int kPartRows = 2;  // rows of a group in flight in the forward pass

// Threads of a workgroup in the forward pass.
__host__ __device__ constexpr int part_threads(int G) { return G < 256 ? 512 : 256; }

template <int DT, int G, int NI, bool SINGLE>
__global__ __launch_bounds__(part_threads(G)) void k_balance_part(BArgs a) {
  typedef typename Row<DT>::T T;
  constexpr int kWork = part_threads(G), kGroups = kWork / G, R = kPartRows;
  constexpr int kSeg = G < 64 ? G : 64;
  extern __shared__ int32_t hist[];                     // [E]
  float* share = reinterpret_cast<float*>(hist + a.E);  // [kGroups][E]
  __shared__ float box[2][G > 64 ? G / 64 * R : 1], far_box[4];
  __shared__ int live_tokens;
  __shared__ double loss_part[kWork / 64];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = G == 64 ? wv : tid / G, c0 = tid % G * 4;
  const int c = blockIdx.x;
  if (!SINGLE && c == 0 && tid == 0) *a.ws_ticket = 0u;
  const int t_end = min(a.M, (c + 1) * a.chunk);
  int t0 = c * a.chunk, filled = 0;
  double loss = 0.0;
  for (int b = SINGLE ? 0 : sequence_of(a, t0); b < a.B && (SINGLE || t0 < t_end); ++b) {
    const int t1 = max(t0, b == a.B - 1 ? t_end : min(offset_of(a, b + 1), t_end));
    if (!SINGLE && t1 == t0) continue;
    Four<DT> next[R][NI];
    int next_mask[R];  // with its row: a load to wait for would drain those in flight
    auto fetch = [&](int t) {  // rows past the sequence's last one repeat it
#pragma unroll
      for (int r = 0; r < R; ++r) next_mask[r] = a.mask ? a.mask[min(t + r, t1 - 1)] : 1;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < NI; ++i)
          next[r][i] = load4<DT>(static_cast<const T*>(a.logits) + (size_t)min(t + r, t1 - 1) * a.E, c0 + i * G * 4, a.E,
                                  i < NI - 1);
    };
    if (t1 > t0) fetch(t0 + grp * R);  // on their way while the ids are counted
    for (int e = tid; e < a.E; e += kWork) hist[e] = 0;
    if (tid == 0) live_tokens = 0;
    __syncthreads();
    for (int i = tid; i < (t1 - t0) * a.k; i += kWork) {
      const int id = a.ids[(size_t)t0 * a.k + i], mask = a.mask ? a.mask[t0 + i / a.k] : 1;
      if (id >= 0 && id < a.E && mask) atomicAdd(&hist[id], 1);
    }
    float acc[NI][4] = {};
    int n = 0, turn = 0;
    for (int tb = t0; tb < t1; tb += R * kGroups, turn ^= 1) {
      const int t = tb + grp * R;
      float s[R][NI][4], total[R];
      bool live[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        live[r] = t + r < t1 && next_mask[r];
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) s[r][i][v] = Row<DT>::get(next[r][i].v[v]);
      }
      if (tb + R * kGroups < t1) fetch(t + R * kGroups);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        total[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            s[r][i][v] = sigmoid(s[r][i][v]);
            total[r] += s[r][i][v];
          }
        total[r] = seg_sum<kSeg>(total[r]);
      }
      if constexpr (G > 64) {
        if (lane == 0)
#pragma unroll
          for (int r = 0; r < R; ++r) box[turn][wv * R + r] = total[r];
        __syncthreads();
        sum_waves<G / 64, R>(box[turn], total);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (!live[r]) continue;
        ++n;
        float inv = 1.0f;
        if (total[r] < kTiny)
          far_shares<DT, G, NI>(static_cast<const T*>(a.logits) + (size_t)(t + r) * a.E, c0, a.E, far_box, s[r]);
        else
          inv = 1.0f / total[r];
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][v] = fmaf(s[r][i][v], inv, acc[i][v]);
      }
    }
    if (kGroups > 1 && tid % G == 0) atomicAdd(&live_tokens, n);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (i < NI - 1 || c0 + i * G * 4 + v < a.E) share[grp * a.E + c0 + i * G * 4 + v] = acc[i][v];
    __syncthreads();  // the histogram is complete as well
    if (kGroups > 1) n = live_tokens;
    auto sum = [&](int e) {  // over the groups, in their order
      float v = share[e];
#pragma unroll
      for (int w = 1; w < kGroups; ++w) v += share[w * a.E + e];
      return v;
    };
    if constexpr (SINGLE) {
      for (int e = tid; e < a.E; e += kWork) {
        const double mean = n > 0 ? (double)sum(e) / n : 0.0;
        a.counts[(size_t)b * a.E + e] = hist[e];
        a.shares[(size_t)b * a.E + e] = (float)mean;
        if (n > 0) loss += (double)hist[e] * mean / n;
      }
      filled += n > 0;
      if (tid == 0) a.tokens[b] = n;
    } else {
      const size_t piece = (size_t)(c + b) * a.E;
      for (int e = tid; e < a.E; e += kWork) {
        a.ws_share[piece + e] = sum(e);
        a.ws_count[piece + e] = hist[e];
      }
      if (tid == 0) a.ws_n[c + b] = n;
    }
    __syncthreads();
    t0 = t1;
  }
  if constexpr (SINGLE) {
    loss = wave_sum(loss);
    if (lane == 0) loss_part[wv] = loss;
    __syncthreads();
    if (tid == 0) {
      loss = loss_part[0];
      for (int w = 1; w < kWork / 64; ++w) loss += loss_part[w];
      a.loss[0] = loss_of(a, loss, filled);
      a.tokens[a.B] = filled;
    }
  }
}

// The tiles' parts of the loss, in their order, by one workgroup.
__device__ __forceinline__ void finish(const BArgs& a, int tiles, double* sh, int* nn) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, waves = blockDim.x / 64;
  double total = 0.0;
  int filled = 0;
#pragma unroll 4
  for (int i = tid; i < tiles * a.B; i += blockDim.x)
    total += __hip_atomic_load(&a.ws_loss[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = tid; i < a.B; i += blockDim.x)
    filled += __hip_atomic_load(&a.tokens[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 0;
  total = wave_sum(total);
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) filled += __shfl_xor(filled, m, 64);
  if (lane == 0) {
    sh[wv] = total;
    nn[wv] = filled;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < waves; ++w) {
      total += sh[w];
      filled += nn[w];
    }
    a.tokens[a.B] = filled;
    a.loss[0] = loss_of(a, total, filled);
  }
}

// A workgroup adds up 2^lcols experts of a sequence, 2^lwalkers threads to an
// expert, each every (walkers)-th piece, eight at a time in flight.  TICKET: the
// workgroup that finishes last adds up the loss, else a third launch does.  LONG:
// 32 walkers and 32 experts, known to the compiler (8192 x 896 forward 15.5 us, as
// arguments 16.0).
template <bool TICKET, bool LONG>
__global__ __launch_bounds__(1024) void k_balance_sum(BArgs a, int lcols, int lwalkers) {
  if constexpr (LONG) lcols = lwalkers = 5;
  __shared__ double sh[1024 + 32];
  __shared__ int ct[1024 + 32], nn[16];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x / 64;
  const int cols = 1 << lcols, walkers = 1 << lwalkers, walker = tid >> lcols, l = tid & (cols - 1);
  const int tiles = gridDim.x, b = blockIdx.y;
  const int ec = min((int)blockIdx.x * cols + l, a.E - 1);
  const int t0 = offset_of(a, b), t1 = b == a.B - 1 ? a.M : offset_of(a, b + 1);
  int first = 0, end = 0;
  if (t1 > t0) {
    first = t0 / a.chunk + b;
    end = (t1 - 1) / a.chunk + b + 1;
  }
  double s = 0.0;
  int count = 0, n = 0;
  for (int p = first + tid; p < end; p += blockDim.x) n += a.ws_n[p];
  for (int p0 = first + walker; p0 < end; p0 += 8 * walkers) {
    float f[8];
    int i[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const size_t at = (size_t)min(p0 + u * walkers, end - 1) * a.E + ec;
      f[u] = a.ws_share[at];
      i[u] = a.ws_count[at];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (p0 + u * walkers < end) {
        s += (double)f[u];
        count += i[u];
      }
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) n += __shfl_xor(n, m, 64);
  sh[walker * (cols + 1) + l] = s;
  ct[walker * (cols + 1) + l] = count;
  if (lane == 0) nn[wv] = n;
  __syncthreads();
  // the walkers of a column lie side by side now, for a butterfly
  const int h = tid & (walkers - 1), col = tid >> lwalkers, ecol = blockIdx.x * cols + col;
  s = sh[h * (cols + 1) + col];
  count = ct[h * (cols + 1) + col];
  for (int m = walkers / 2; m >= 1; m >>= 1) {
    s += __shfl_xor(s, m, 64);
    count += __shfl_xor(count, m, 64);
  }
  n = nn[0];
  for (int w = 1; w < waves; ++w) n += nn[w];
  const double share = n > 0 ? s / n : 0.0;
  const bool mine = h == 0 && ecol < a.E;
  if (mine) {
    a.counts[(size_t)b * a.E + ecol] = count;
    a.shares[(size_t)b * a.E + ecol] = (float)share;
  }
  double part = wave_sum(mine && n > 0 ? (double)count * share / n : 0.0);
  __syncthreads();
  if (lane == 0) sh[wv] = part;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < waves; ++w) part += sh[w];
    a.ws_loss[(size_t)b * tiles + blockIdx.x] = part;
    if (blockIdx.x == 0) a.tokens[b] = n;
    if constexpr (TICKET) {
      last = __hip_atomic_fetch_add(a.ws_ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
             (uint32_t)tiles * (uint32_t)a.B - 1u;
    }
  }
  if constexpr (TICKET) {
    __syncthreads();
    if (last) finish(a, tiles, sh, nn);
  }
}

__global__ __launch_bounds__(1024) void k_balance_loss(BArgs a, int tiles) {
  __shared__ double sh[16];
  __shared__ int nn[16];
  finish(a, tiles, sh, nn);
}

// No token: zeros, one workgroup.
__global__ __launch_bounds__(256) void k_balance_none(BArgs a) {
  for (size_t i = threadIdx.x; i < (size_t)a.B * a.E; i += 256) {
    a.counts[i] = 0;
    a.shares[i] = 0.0f;
  }
  for (int i = threadIdx.x; i <= a.B; i += 256) a.tokens[i] = 0;
  if (threadIdx.x == 0) a.loss[0] = 0.0f;
}

// The gradient that a row's routing weights give the logit of this lane's pick:
// xk its logit (-infinity: no pick), gw its weight's gradient.
template <int S>
__device__ __forceinline__ float pick_grad(float xk, float gw) {
  // scores relative to exp(min(max x, 0)), so they never all underflow
  const float m = fminf(seg_max<S>(xk), 0.0f);
  const float u = fast_exp(-__builtin_fabsf(xk)), q = fast_rcp(1.0f + u);
  float w = xk > 0.0f ? q : (xk != xk ? xk : fast_exp(xk - m) * q);  // s / exp(m)
  const float rest = xk > 0.0f ? u * q : q;                          // 1 - s
  if (m == -__builtin_inff()) w = xk != xk ? xk : 0.0f;  // the maximum passes NaN over
  const float sum = seg_sum<S>(w);
  w = sum > 0.0f || sum != sum ? w / sum : 0.0f;
  return w * rest * (gw - seg_sum<S>(gw * w));
}

// Weights of tokens whose picks all lie below kFar, where their FP32 scores are
// subnormal or zero and the route's quotient is coarse, infinite or 0 / 0: sigmoid
// and exp agree far past FP32 there, so exp(x - max) / sum is the quotient.  From
// kFar up the sum is a normal number (exp(-87) > 2^-126) and nothing is written.
// One read of the ids and a gather of their logits: 8192 x 16 picks of 896 experts
// in 2.2 us, bound by the launch and two round trips (131072 x 32 picks in 17 us).
constexpr float kFar = -87.0f;
constexpr int kFarGrid = 2048;  // workgroups at most; they walk the tokens

template <int DT, int S>
__global__ __launch_bounds__(kThreads) void k_far_weights(BArgs a) {
  constexpr int kTokens = kThreads / S;  // S lanes a token
  const int j = threadIdx.x % S;
  for (int t0 = blockIdx.x * kTokens; t0 < a.M; t0 += gridDim.x * kTokens) {
    const int t = t0 + threadIdx.x / S;
    const bool mine = t < a.M && j < a.k;
    const int id = mine ? a.ids[(size_t)t * a.k + j] : -1;
    float x = -__builtin_inff();
    if (id >= 0 && id < a.E)
      x = Row<DT>::get(static_cast<const typename Row<DT>::T*>(a.logits)[(size_t)t * a.E + id]);
    const float m = seg_max<S>(x);
    if (m < kFar) {  // the same in all lanes of a token
      float w = m > -__builtin_inff() ? fast_exp(x - m) : (x != x ? x : 0.0f);
      const float sum = seg_sum<S>(w);
      w = sum > 0.0f || sum != sum ? w / sum : 0.0f;
      if (mine) static_cast<float*>(a.out)[(size_t)t * a.k + j] = w;
    }
  }
}

// Token t's mask, 1 without one: a load either way, since a constant in its place
// waits for the loads in flight before it is written over the last one's register
// (16384 x 4096 FP32 without a mask 101 us, with the constant 108).
__device__ __forceinline__ int mask_of(const BArgs& a, int t) {
  const uint8_t* p = a.mask ? a.mask + t : reinterpret_cast<const uint8_t*>(a.ids);
  return *p | (a.mask ? 0 : 1);
}

// d/dx of the balance loss of row t: g_b s' / S * (count[b,e] - sum_e' count[b,e'] p[e']),
// g_b = grad_loss coef E / (k n_b^2 B'); of the picks' weights:
// w_j (1 - s_j) (grad_w_j - sum_i grad_w_i w_i), added through a row of LDS.  One
// row a group is in flight: with two, fewer workgroups fit (16384 x 4096 FP32 109 and
// 102 us, 8192 x 896 BF16 12.4 and 11.7).
template <int DT, int G, int NI>
__global__ __launch_bounds__(kThreads) void k_router_backward(BArgs a) {
  typedef typename Row<DT>::T T;
  constexpr int kGroups = kThreads / G, kSeg = G < 64 ? G : 64;
  extern __shared__ float picks[];  // [kGroups][E], zero between rows
  __shared__ float box[2][G > 64 ? G / 64 : 1], far_box[4];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = G == 64 ? wv : tid / G, c0 = tid % G * 4;
  float* extra = picks + (size_t)grp * a.E;
  const int c = blockIdx.x;
  const int t_end = min(a.M, (c + 1) * a.chunk);
  int t0 = c * a.chunk;
  const float gl = a.grad_loss ? *a.grad_loss : 1.0f;
  const int filled = a.counts ? a.tokens[a.B] : 0;
  // picks: up to 16 of them, in the first 16 lanes of the group's first wave
  // (groups of 16 have no more picks); more, in the whole wave
  const bool few = G == 16 || a.k <= 16;
  const int j = few ? lane % 16 : lane;
  const bool picker = j < a.k && (G > 64 ? wv == 0 : true) && (!few || G == 16 || lane < 16);
  bool fresh = true;
  for (int b = sequence_of(a, t0); b < a.B && t0 < t_end; ++b) {
    const int t1 = b == a.B - 1 ? t_end : min(offset_of(a, b + 1), t_end);
    if (t1 <= t0) continue;
    Four<DT> next[NI];
    auto fetch = [&](int t) {  // rows past the sequence's last one repeat it
      if (a.counts)
#pragma unroll
        for (int i = 0; i < NI; ++i)
          next[i] = load4<DT>(static_cast<const T*>(a.logits) + (size_t)min(t, t1 - 1) * a.E, c0 + i * G * 4, a.E,
                              i < NI - 1);
    };
    // a row's ids are two rows ahead, the logits that they name one
    int mask, next_mask;  // of the same rows: a load to wait for would drain those in flight
    int id, next_id;
    float gw, next_gw;
    T xk;
    auto fetch_ids = [&](int t) {
      next_mask = mask_of(a, min(t, t1 - 1));
      next_id = -1;
      if (a.grad_w && picker && t < t1) {
        next_id = a.ids[(size_t)t * a.k + j];
        next_gw = a.grad_w[(size_t)t * a.k + j];
      }
    };
    auto fetch_picks = [&](int t) {  // of the row whose ids have come, and the next one's ids
      mask = next_mask;
      if (a.grad_w) {
        id = mask && next_id < a.E ? next_id : -1;
        gw = id >= 0 ? next_gw : 0.0f;
        xk = Row<DT>::put(-__builtin_inff());
        if (id >= 0) xk = static_cast<const T*>(a.logits)[(size_t)t * a.E + id];
      }
      fetch_ids(t + kGroups);
    };
    fetch_ids(t0 + grp);
    fetch(t0 + grp);
    float cnt[NI][4] = {}, g = 0.0f;
    if (a.counts) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (i < NI - 1 || c0 + i * G * 4 + v < a.E) cnt[i][v] = (float)a.counts[(size_t)b * a.E + c0 + i * G * 4 + v];
      const int n = a.tokens[b];
      if (n > 0 && filled > 0)
        g = (float)((double)gl * a.coef * a.E / ((double)a.k * n * (double)n * filled));
    }
    if (a.grad_w) {
      if (fresh) {
        for (int i = tid; i < kGroups * a.E; i += kThreads) picks[i] = 0.0f;
        __syncthreads();
      }
    }
    fetch_picks(t0 + grp);
    fresh = false;
    for (int tb = t0; tb < t1; tb += kGroups) {
      const int t = tb + grp;
      const T* row = static_cast<const T*>(a.logits) + (size_t)min(t, t1 - 1) * a.E;
      float d[NI][4], total = 0.0f, dot = 0.0f, p = 0.0f;
      int at = -1;  // the pick's place in LDS
      if (a.grad_w) {
        at = id;
        const float x = Row<DT>::get(xk);
        p = few ? pick_grad<16>(x, gw) : pick_grad<64>(x, gw);
      }
      const bool live = t < t1 && mask;
      if (a.counts)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) d[i][v] = Row<DT>::get(next[i].v[v]);
      if (tb + kGroups < t1) {
        fetch_picks(t + kGroups);
        fetch(t + kGroups);
      }
      if (at >= 0) atomicAdd(&extra[at], p);
      if (a.counts) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float s = sigmoid(d[i][v], d[i][v]);
            total += s;
            dot = fmaf(cnt[i][v], s, dot);
          }
        total = seg_sum<kSeg>(total);
        dot = seg_sum<kSeg>(dot);
        if constexpr (G > 64) {
          if (lane == 0) {
            box[0][wv] = total;
            box[1][wv] = dot;
          }
        }
      }
      if constexpr (G > 64) {
        __syncthreads();
        if (a.counts) {
          total = dot = 0.0f;
#pragma unroll
          for (int w = 0; w < G / 64; ++w) {
            total += box[0][w];
            dot += box[1][w];
          }
        }
      } else {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      if (t < t1) {
        float f = 0.0f, mean = 0.0f;
        if (live && a.counts) {
          float scale = 1.0f;
          if (total < kTiny) {
            far_shares<DT, G, NI>(row, c0, a.E, far_box, d);
            dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
              for (int v = 0; v < 4; ++v) dot = fmaf(cnt[i][v], d[i][v], dot);
            dot = group_sum<G>(dot, far_box);
          } else {
            scale = 1.0f / total;
          }
          f = g * scale;
          mean = dot * scale * f;
        }
        T* dst = static_cast<T*>(a.out) + (size_t)t * a.E;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          const int col = c0 + i * G * 4;
          if (live && a.counts)
#pragma unroll
            for (int v = 0; v < 4; ++v) o[v] = fmaf(cnt[i][v], f, -mean) * d[i][v];
          if (live && a.grad_w)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (i < NI - 1 || col + v < a.E) o[v] += extra[col + v];
          store4<DT>(dst, col, a.E, i < NI - 1, o);
        }
      }
      if constexpr (G > 64) __syncthreads();
      else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (at >= 0) extra[at] = 0.0f;
    }
    t0 = t1;
  }
}

size_t align16(size_t v) { return (v + 15) & ~size_t(15); }

// Threads that share a row: sixteen lanes while sixteen columns a lane hold it,
// then a wave, then four.  (With four columns a thread and up to 1024 threads a
// row, the sums over the lanes cost a quarter of the arithmetic and a barrier of
// sixteen waves held the loads back: 8192 x 896 backward 19 us, 16384 x 4096 150.)
// A whole wave for 128 experts left half its lanes idle and paid its sums per row:
// 131072 x 128 forward 50 us against 20, backward 64 against 24.  Sixteen lanes have
// no room for more than sixteen picks, a lane each.
int group_of(int E, bool picks, int k) { return E <= 256 && !(picks && k > 16) ? 16 : E <= 1024 ? 64 : 256; }
int columns_of(int E, int G) { return (E + 4 * G - 1) / (4 * G); }

constexpr int kSingleBatches = 4;  // batches that one workgroup does alone
constexpr int kSingleB = 4;  // 64 x 64: one workgroup 7.0 us for 3 sequences, 11.9 for 6, several 10.4
// Workgroups of the second kernel that may share a counter, 40 ns each, in place of
// a third launch (65536 x 64, 64 sequences: with 64 of them 18.9 us, with the launch
// 17.8; 65536 x 128, 16 sequences, 32 of them: 17.2 and 18.2).
constexpr int kTicketMax = 32;

// Tokens of a workgroup when `grid` of them run at once.  It takes its sequences one
// after another, 2 us each: fewer rows where they are short (forward 256 x 256, 8
// sequences 19.3 -> 13.4 us; 901 x 190, 49 of them 28 -> 15.8; 2000 x 64, 200 of them 32.5 ->
// 15.1; backward the last two 12.8 -> 8.6 and 11.8 -> 7.8).
int chunk_of(int M, int B, int batch, int grid) {
  const int each = (M + grid - 1) / grid;
  if (each > batch) return (each + batch - 1) / batch * batch;
  int chunk = batch;
  while (chunk > 4 && chunk > M / B / 4 && M / chunk < grid) chunk /= 2;
  return chunk;
}

struct Plan {
  int chunk, chunks, lcols, lwalkers, tiles;
  bool single;
  size_t share, count, n, loss, ticket, total;
};

Plan plan_of(int M, int E, int B) {
  Plan p{};
  const int G = group_of(E, false, 0), batch = kPartRows * (part_threads(G) / G), alone = kSingleBatches * batch;
  p.single = M <= alone && B <= kSingleB;
  // a workgroup for each compute unit: eight waves, or twice four
  p.chunk = p.single ? alone : chunk_of(M, B, batch, G < 256 ? 256 : 512);
  p.chunks = (M + p.chunk - 1) / p.chunk;
  const int pieces = p.chunks / B;  // of a sequence
  // Threads of the second kernel: 32 walkers of 32 experts for long sequences (1024
  // threads), else 256 threads, 8 walkers or 4 when each of eight would get less than
  // four pieces of an average sequence (us, 8 / 4 walkers: 16384 x 4096, 37 equal
  // sequences 67 / 61; 8192 x 896, 128 of them 26.7 / 23.2, and where one of these has
  // 90 % of the tokens 32.1 / 30.5).  2 walkers only shorten a launch of many
  // workgroups, one sequence's chain of pieces takes the longer (4 / 2 walkers: 16384
  // x 4096, 200 sequences 84 / 72, with one of 95 % 95 / 91; the 8192 x 896 above 23.2
  // / 22.0 and 30.5 / 33.5).
  p.lcols = 5;
  p.lwalkers = pieces >= 64 ? 5 : 3;
  p.tiles = (E + 31) / 32;
  while (p.lwalkers < 5 && p.lwalkers > 1 && (1 << p.lcols) < E && pieces < 4 << p.lwalkers &&
         (p.lwalkers > 2 || (int64_t)p.tiles * B > 4096)) {
    ++p.lcols;
    --p.lwalkers;
    p.tiles = (E + (1 << p.lcols) - 1) >> p.lcols;
  }
  const size_t all = (size_t)p.chunks + B;
  p.share = 0;
  p.count = p.share + align16(all * E * 4);
  p.n = p.count + align16(all * E * 4);
  p.loss = p.n + align16(all * 4);
  p.ticket = p.loss + align16((size_t)B * p.tiles * 8);
  p.total = p.ticket + 16;
  return p;
}

bool valid_sizes(int M, int E, int k, int B) {
  return M >= 0 && E >= 1 && E <= 4096 && k >= 1 && k <= 64 && B >= 1 && B <= 65535;
}

// Token and route numbers, and a chunk past the last token, in 32 bits.
bool fits(int M, int k) { return M <= (1 << 30) && (int64_t)M * k <= INT32_MAX; }

enum { kPart, kSingle, kBack };

template <int WHAT, int DT, int G, int NI>
const void* one() {
  if constexpr (WHAT == kBack) return reinterpret_cast<const void*>(k_router_backward<DT, G, NI>);
  else return reinterpret_cast<const void*>(k_balance_part<DT, G, NI, WHAT == kSingle>);
}
template <int WHAT, int DT>
const void* kernel_of(int E, int G) {
  const int ni = columns_of(E, G);
  if (G == 16) {
    switch (ni) {
      case 1: return one<WHAT, DT, 16, 1>();
      case 2: return one<WHAT, DT, 16, 2>();
      case 3: return one<WHAT, DT, 16, 3>();
      default: return one<WHAT, DT, 16, 4>();
    }
  }
  if (G == 64) {
    switch (ni) {
      case 1:
        if constexpr (WHAT == kBack) return one<WHAT, DT, 64, 1>();  // more than sixteen picks
        [[fallthrough]];
      case 2: return one<WHAT, DT, 64, 2>();
      case 3: return one<WHAT, DT, 64, 3>();
      default: return one<WHAT, DT, 64, 4>();
    }
  }
  switch (ni) {
    case 2: return one<WHAT, DT, 256, 2>();
    case 3: return one<WHAT, DT, 256, 3>();
    default: return one<WHAT, DT, 256, 4>();
  }
}
template <int WHAT>
const void* kernel_of(int dtype, int E, int G) {
  return dtype == MRS_DTYPE_F32 ? kernel_of<WHAT, MRS_DTYPE_F32>(E, G) : kernel_of<WHAT, MRS_DTYPE_BF16>(E, G);
}

const void* sum_kernel(bool ticket, bool many) {
  if (ticket)
    return many ? reinterpret_cast<const void*>(k_balance_sum<true, true>)
                : reinterpret_cast<const void*>(k_balance_sum<true, false>);
  return many ? reinterpret_cast<const void*>(k_balance_sum<false, true>)
              : reinterpret_cast<const void*>(k_balance_sum<false, false>);
}

int launch(const void* fn, dim3 grid, int threads, size_t lds, BArgs& a, void* stream) {
  void* params[] = {&a};
  return hipLaunchKernel(fn, grid, dim3(threads), params, lds, reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? MRS_OK
             : MRS_ERR_LAUNCH;
}

}  // namespace

extern "C" size_t moe_balance_workspace_bytes(int M, int E, int k, int B) {
  if (!valid_sizes(M, E, k, B) || !fits(M, k)) return (size_t)-1;
  return plan_of(M, E, B).total;
}

extern "C" int moe_balance_loss(const void* logits, int logits_dtype, const int32_t* ids, const int32_t* seq_offsets,
                                const uint8_t* mask, int M, int E, int k, int B, float coef, float* loss,
                                int32_t* counts, int32_t* tokens, float* shares, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!valid_sizes(M, E, k, B) || (!seq_offsets && B != 1) ||
      (logits_dtype != MRS_DTYPE_F32 && logits_dtype != MRS_DTYPE_BF16))
    return MRS_ERR_INVALID_ARG;
  if (!fits(M, k)) return MRS_ERR_OVERFLOW;
  if (!loss || !counts || !tokens || !shares) return MRS_ERR_NULL_POINTER;
  if (!aligned(loss, 4) || !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(shares, 4))
    return MRS_ERR_MISALIGNED;
  Plan p = plan_of(M, E, B);
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
  a.coef = coef;
  a.loss = loss;
  a.counts = counts;
  a.tokens = tokens;
  a.shares = shares;
  if (M == 0) return launch(reinterpret_cast<const void*>(k_balance_none), dim3(1), 256, 0, a, stream);
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
  const int G = group_of(E, false, k), threads = part_threads(G);
  const size_t lds = (size_t)E * 4 * (1 + threads / G);
  if (p.single) return launch(kernel_of<kSingle>(logits_dtype, E, G), dim3(1), threads, lds, a, stream);
  int rc = launch(kernel_of<kPart>(logits_dtype, E, G), dim3(p.chunks), threads, lds, a, stream);
  if (rc != MRS_OK) return rc;
  const bool ticket = (int64_t)p.tiles * B <= kTicketMax;
  void* sum_params[] = {&a, &p.lcols, &p.lwalkers};
  if (hipLaunchKernel(sum_kernel(ticket, p.lwalkers == 5), dim3(p.tiles, B), dim3(1 << (p.lcols + p.lwalkers)), sum_params,
                      0, reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
    return MRS_ERR_LAUNCH;
  if (ticket) return MRS_OK;
  int tiles = p.tiles;
  void* params[] = {&a, &tiles};
  return hipLaunchKernel(reinterpret_cast<const void*>(k_balance_loss), dim3(1), dim3(1024), params, 0,
                         reinterpret_cast<hipStream_t>(stream)) == hipSuccess
             ? MRS_OK
             : MRS_ERR_LAUNCH;
}

extern "C" int moe_router_backward(const void* logits, int logits_dtype, const int32_t* ids, const float* grad_w,
                                   const int32_t* counts, const int32_t* tokens, const float* grad_loss,
                                   const int32_t* seq_offsets, const uint8_t* mask, int M, int E, int k, int B,
                                   float coef, void* grad_logits, void* stream) {
  if (!valid_sizes(M, E, k, B) || (!seq_offsets && B != 1) ||
      (logits_dtype != MRS_DTYPE_F32 && logits_dtype != MRS_DTYPE_BF16))
    return MRS_ERR_INVALID_ARG;
  if (!fits(M, k)) return MRS_ERR_OVERFLOW;
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
  const int G = group_of(E, grad_w != nullptr, k);
  a.chunk = chunk_of(M, B, kThreads / G, 1024);  // four workgroups a compute unit
  a.coef = coef;
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.grad_w = grad_w;
  a.grad_loss = grad_loss;
  a.out = grad_logits;
  const size_t lds = grad_w ? (size_t)(kThreads / G) * E * 4 : 0;
  return launch(kernel_of<kBack>(logits_dtype, E, G), dim3((M + a.chunk - 1) / a.chunk), kThreads, lds, a, stream);
}

extern "C" int moe_route_far_weights(const void* logits, int logits_dtype, const int32_t* ids, int M, int E, int k,
                                     float* weights, void* stream) {
  if (!valid_sizes(M, E, k, 1) || (logits_dtype != MRS_DTYPE_F32 && logits_dtype != MRS_DTYPE_BF16))
    return MRS_ERR_INVALID_ARG;
  if (!fits(M, k)) return MRS_ERR_OVERFLOW;
  if (M == 0) return MRS_OK;
  if (!logits || !ids || !weights) return MRS_ERR_NULL_POINTER;
  if (!aligned(logits, logits_dtype == MRS_DTYPE_F32 ? 4 : 2) || !aligned(ids, 4) || !aligned(weights, 4))
    return MRS_ERR_MISALIGNED;
  BArgs a{};
  a.logits = logits;
  a.ids = ids;
  a.M = M;
  a.E = E;
  a.k = k;
  a.out = weights;
  const int S = k <= 16 ? 16 : 64, tokens = kThreads / S;
  const bool f32 = logits_dtype == MRS_DTYPE_F32;
  const void* fn = S == 16 ? (f32 ? reinterpret_cast<const void*>(k_far_weights<MRS_DTYPE_F32, 16>)
                                  : reinterpret_cast<const void*>(k_far_weights<MRS_DTYPE_BF16, 16>))
                           : (f32 ? reinterpret_cast<const void*>(k_far_weights<MRS_DTYPE_F32, 64>)
                                  : reinterpret_cast<const void*>(k_far_weights<MRS_DTYPE_BF16, 64>));
  const int grid = (M + tokens - 1) / tokens;
  return launch(fn, dim3(grid < kFarGrid ? grid : kFarGrid), kThreads, 0, a, stream);
}
