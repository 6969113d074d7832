// Balance loss of the router with per-expert counts, and the gradient of the
// router's logits (C ABI: include/flint_moe_balance.h).
//
// One pass over the logits each way. With f_be - 1 = (E c_be - k T_b) / (k T_b)
// (whole numbers until the division, so nothing cancels) and sum_e p_te = 1,
//   sum_e f_be p_te = 1 + F_t,   F_t = sum_e (f_be - 1) s_te / sum_e s_te
//   loss = alpha / n_seq  sum_t (1 + F_t) / T_b
//   dz_tj = dloss alpha / (n_seq T_b) p_tj ((f_bj - 1) - F_t) (1 - s_tj)
// so a row needs two sums, sum_e s and sum_e (f - 1) s, and no second look at
// memory: the counts come first, from the picks alone.
//
// One warp per token row, 16-byte loads. Both kernels move T E floats and are
// bound by memory bandwidth.
#include <algorithm>

#include "common.cuh"
#include "flint_moe_balance.h"

namespace flint {
namespace bal {

constexpr int MAX_E = MAX_EXPERTS;

struct BalArgs {
  int T, E, k, n_seq, renorm;
  float routed_scale, alpha;
  const float* logits;
  const int* idx;
  const int* seq_start;  // or null: one sequence of T tokens
  float* loss;
  int* counts;
  int* seq_counts;
  int* seq_tokens;
  double* partial;  // [gridDim.x of the loss kernel]
  unsigned* ticket;
  const float* dloss;
  const float* dw;
  float* dlogits;
};

// First token of sequence b, kept within [0, T] whatever the array holds.
__device__ __forceinline__ int seq_at(const BalArgs& a, int b) {
  if (!a.seq_start) return b == 0 ? 0 : a.T;
  return min(max(__ldg(a.seq_start + b), 0), a.T);
}

// Sequence of token t: the last b with seq_start[b] <= t (so an empty sequence
// is never found), -1 before the first, n_seq behind the last.
__device__ __forceinline__ int seq_of(const BalArgs& a, int t) {
  if (!a.seq_start) return 0;
  int lo = -1, hi = a.n_seq;  // seq_at(lo) <= t < seq_at(hi + 1), in bounds for any contents
  if (seq_at(a, a.n_seq) <= t) return a.n_seq;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (seq_at(a, m) <= t)
      lo = m;
    else
      hi = m;
  }
  return lo;
}

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// s = sigmoid(z) and q = 1 - s without cancellation: with e = exp(-z), s = 1 / (1 + e) and
// q = e s. e is held at 1e37, where s is still an FP32 normal; rows in which no s is above
// 1e-30 take the exact shares below instead.
constexpr float LOW_ROW = 1e-30f;
__device__ __forceinline__ void sigmoid2(float z, float& s, float& q) {
  const float e = fminf(__expf(-z), 1e37f);
  s = __fdividef(1.0f, 1.0f + e);
  q = e * s;
}

// A row's logits: lane l holds elements 4 (l + 32 i) .. + 3 (VEC, E % 4 == 0) or l + 32 i.
template <bool VEC>
__device__ __forceinline__ int elem(int lane, int j) {
  return VEC ? 4 * (lane + 32 * (j >> 2)) + (j & 3) : lane + 32 * j;
}

template <int PER, bool VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float (&z)[PER]) {
  if (VEC) {
#pragma unroll
    for (int i = 0; i < PER / 4; ++i) {
      const int e = 4 * (lane + 32 * i);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (e < E) v = __ldg(reinterpret_cast<const float4*>(row + e));
      z[4 * i] = v.x;
      z[4 * i + 1] = v.y;
      z[4 * i + 2] = v.z;
      z[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) z[j] = lane + 32 * j < E ? __ldg(row + lane + 32 * j) : 0.f;
  }
}

// s (the row's scores, or for a low row exp(z - max z), which has the same shares) and
// q = 1 - sigmoid(z) of this lane's elements, and the row's sum of s.
template <int PER, bool VEC>
__device__ __forceinline__ float scores(const float (&z)[PER], int E, int lane, float (&s)[PER], float (&q)[PER]) {
  float S = 0.f;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const bool in = elem<VEC>(lane, j) < E;
    sigmoid2(z[j], s[j], q[j]);
    if (!in) s[j] = q[j] = 0.f;
    S += s[j];
  }
  S = warp_sum(S);
  if (S < LOW_ROW * E) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (elem<VEC>(lane, j) < E) m = fmaxf(m, z[j]);
    m = warp_max(m);
    float acc = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      s[j] = elem<VEC>(lane, j) < E && m > -INFINITY ? __expf(z[j] - m) : 0.f;
      acc += s[j];
    }
    S = warp_sum(acc);
  }
  return S;
}

// f - 1 of this lane's experts in sequence b.
template <int PER, bool VEC>
__device__ __forceinline__ void load_f(const BalArgs& a, int b, int Tb, int lane, float (&f)[PER]) {
  const int* c = a.seq_counts + (size_t)b * a.E;
  const long long even = (long long)a.k * Tb;
  const float inv = even > 0 ? 1.0f / (float)even : 0.f;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = elem<VEC>(lane, j);
    f[j] = e < a.E ? (float)((long long)__ldcg(c + e) * a.E - even) * inv : 0.f;
  }
}

__global__ void __launch_bounds__(256) k_bal_zero(const BalArgs a) {
  const size_t n = (size_t)a.n_seq * a.E;
  for (size_t i = blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) a.seq_counts[i] = 0;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < a.n_seq; i += gridDim.x * 256) a.seq_tokens[i] = 0;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < a.E; i += gridDim.x * 256) a.counts[i] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *a.ticket = 0;
    if (a.T == 0) *a.loss = 0.f;
  }
}

__global__ void __launch_bounds__(256) k_bal_count(const BalArgs a) {
  for (int t = blockIdx.x * 256 + threadIdx.x; t < a.T; t += gridDim.x * 256) {
    const int b = seq_of(a, t);
    const int* p = a.idx + (size_t)t * a.k;
    if (b < 0 || b >= a.n_seq || __ldg(p) < 0) continue;
    atomicAdd(a.seq_tokens + b, 1);
    for (int j = 0; j < a.k; ++j) {
      const int e = __ldg(p + j);
      if (e < 0 || e >= a.E) continue;
      atomicAdd(a.seq_counts + (size_t)b * a.E + e, 1);
      atomicAdd(a.counts + e, 1);
    }
  }
}

// Sum over the block's tokens of (1 + F_t) / T_b in FP64; the last block to finish adds the
// blocks' sums in block order.
template <int PER, bool VEC>
__global__ void __launch_bounds__(256) k_bal_loss(const BalArgs a) {
  __shared__ double red[8];
  __shared__ bool last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (a.T + gridDim.x * 8 - 1) / (gridDim.x * 8);  // consecutive tokens of a warp
  const int t0 = min(a.T, (blockIdx.x * 8 + warp) * per), t1 = min(a.T, t0 + per);
  double acc = 0.0;
  int b = -2, Tb = 0;
  int b_end = -1;
  float f[PER];
  for (int t = t0; t < t1; ++t) {
    if (t >= b_end) {
      b = seq_of(a, t);
      b_end = b < 0 ? seq_at(a, 0) : (b < a.n_seq ? seq_at(a, b + 1) : a.T);
      b_end = max(b_end, t + 1);
      if (b >= 0 && b < a.n_seq) {
        Tb = __ldcg(a.seq_tokens + b);
        load_f<PER, VEC>(a, b, Tb, lane, f);
      }
    }
    if (b < 0 || b >= a.n_seq || __ldg(a.idx + (size_t)t * a.k) < 0) continue;
    float z[PER], s[PER], q[PER];
    load_row<PER, VEC>(a.logits + (size_t)t * a.E, a.E, lane, z);
    const float S = scores<PER, VEC>(z, a.E, lane, s, q);
    float F = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) F = fmaf(f[j], s[j], F);
    F = warp_sum(F);
    if (S > 0.f) acc += (1.0 + (double)(F / S)) / (double)Tb;
  }
  if (lane == 0) red[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int w = 0; w < 8; ++w) v += red[w];
    a.partial[blockIdx.x] = v;
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last || warp != 0) return;
  __threadfence();
  double v = 0.0;
  for (int i = lane; i < (int)gridDim.x; i += 32) v += __ldcg(a.partial + i);
  v = warp_sum_d(v);
  if (lane == 0) *a.loss = (float)(v * ((double)a.alpha / (double)a.n_seq));
}

template <int PER, bool VEC>
__global__ void __launch_bounds__(256) k_bal_backward(const BalArgs a) {
  __shared__ float extra_s[8][MAX_E];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (a.T + gridDim.x * 8 - 1) / (gridDim.x * 8);
  const int t0 = min(a.T, (blockIdx.x * 8 + warp) * per), t1 = min(a.T, t0 + per);
  float* extra = extra_s[warp];  // routing-weight part of the row's gradient, zero but at its picks
  for (int e = lane; e < MAX_E; e += 32) extra[e] = 0.f;
  __syncwarp();
  const float up = (a.dloss ? __ldg(a.dloss) : 1.0f) * (a.alpha / (float)a.n_seq);
  int b = -2, b_end = -1;
  float c = 0.f;
  float f[PER];
  for (int t = t0; t < t1; ++t) {
    if (t >= b_end) {
      b = seq_of(a, t);
      b_end = b < 0 ? seq_at(a, 0) : (b < a.n_seq ? seq_at(a, b + 1) : a.T);
      b_end = max(b_end, t + 1);
      if (b >= 0 && b < a.n_seq) {
        const int Tb = __ldcg(a.seq_tokens + b);
        load_f<PER, VEC>(a, b, Tb, lane, f);
        c = Tb > 0 ? up / (float)Tb : 0.f;
      }
    }
    if (b < 0 || b >= a.n_seq) continue;
    const float* row = a.logits + (size_t)t * a.E;
    float* out = a.dlogits + (size_t)t * a.E;
    const int* p = a.idx + (size_t)t * a.k;
    const bool counted = __ldg(p) >= 0;
    float d[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) d[j] = 0.f;
    if (counted) {
      float z[PER], s[PER], q[PER];
      load_row<PER, VEC>(row, a.E, lane, z);
      const float S = scores<PER, VEC>(z, a.E, lane, s, q);
      float F = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) F = fmaf(f[j], s[j], F);
      F = warp_sum(F);
      const float inv = S > 0.f ? 1.0f / S : 0.f;
      F *= inv;
      const float ci = c * inv;
#pragma unroll
      for (int j = 0; j < PER; ++j) d[j] = (ci * s[j]) * ((f[j] - F) * q[j]);
      if (a.dw) {
        const int e = lane < a.k ? __ldg(p + lane) : -1;
        const bool in = e >= 0 && e < a.E;
        float sp = 0.f, qp = 0.f, g = 0.f;
        if (in) {
          g = __ldg(a.dw + (size_t)t * a.k + lane);
          const float zp = __ldg(row + e);
          sigmoid2(zp, sp, qp);
        }
        float add;
        if (a.renorm) {
          float W = warp_sum(sp);
          if (W < LOW_ROW * MAX_TOPK) {  // every pick's score underflows: the same shares from exp(z - max z)
            const float zp = in ? __ldg(row + e) : -INFINITY;
            const float m = warp_max(zp);
            sp = in && m > -INFINITY ? __expf(zp - m) : 0.f;
            W = warp_sum(sp);
          }
          const float w = W > 0.f ? sp / W : 0.f;
          const float D = warp_sum(in ? g * w : 0.f);
          add = a.routed_scale * w * (g - D) * qp;
        } else {
          add = a.routed_scale * sp * g * qp;
        }
        // An expert picked twice: the picks' parts are added in pick order.
        const unsigned same = __match_any_sync(0xffffffffu, in ? e : -1 - lane);
        float sum = add;
        if (__any_sync(0xffffffffu, same != (1u << lane))) {
          sum = 0.f;
          for (int j = 0; j < a.k; ++j) {
            const float v = __shfl_sync(0xffffffffu, add, j);
            if ((same >> j) & 1u) sum += v;
          }
        }
        if (in) extra[e] = sum;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int el = elem<VEC>(lane, j);
          if (el < a.E) d[j] += extra[el];
        }
        __syncwarp();
        if (in) extra[e] = 0.f;
        __syncwarp();
      }
    }
    if (VEC) {
#pragma unroll
      for (int i = 0; i < PER / 4; ++i) {
        const int e = 4 * (lane + 32 * i);
        if (e < a.E) *reinterpret_cast<float4*>(out + e) = make_float4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (lane + 32 * j < a.E) out[lane + 32 * j] = d[j];
    }
  }
}

}  // namespace bal
}  // namespace flint

using namespace flint;
using namespace flint::bal;

namespace {

constexpr int LOSS_BLOCKS = 152 * 8;  // 8 blocks of 8 warps on each of the 152 SMs

struct BalWs {
  size_t ticket, partial, total;
};
BalWs bal_ws() {
  BalWs w;
  w.ticket = 0;
  w.partial = 256;
  w.total = ws_align(256 + sizeof(double) * LOSS_BLOCKS);
  return w;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool overlap(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np;
}

flint_moe_status check_sizes(const flint_moe_config* c, int32_t T, const int32_t* seq_start, int32_t n_seq, float alpha) {
  const flint_moe_status st = flint_moe_check_config(c);
  if (st != FLINT_MOE_OK) return st;
  if (T < 0 || T > FLINT_MOE_BALANCE_MAX_TOKENS || n_seq < 1 || n_seq > FLINT_MOE_BALANCE_MAX_SEQS) return FLINT_MOE_EINVAL;
  if (!seq_start && n_seq != 1) return FLINT_MOE_EINVAL;
  if (!(alpha >= -3.0e38f && alpha <= 3.0e38f)) return FLINT_MOE_EINVAL;
  return FLINT_MOE_OK;
}

// One warp per token while tokens are few, and no more blocks than LOSS_BLOCKS.
int row_blocks(int T) { return std::max(1, std::min((T + 7) / 8, LOSS_BLOCKS)); }

}  // namespace

extern "C" size_t flint_moe_balance_workspace_bytes(const flint_moe_config* c, int32_t max_tokens, int32_t max_seqs) {
  if (flint_moe_check_config(c) != FLINT_MOE_OK) return 0;
  if (max_tokens < 1 || max_tokens > FLINT_MOE_BALANCE_MAX_TOKENS || max_seqs < 1 || max_seqs > FLINT_MOE_BALANCE_MAX_SEQS)
    return 0;
  return bal_ws().total;
}

extern "C" flint_moe_status flint_moe_balance(const flint_moe_config* c, const float* logits, const int32_t* idx, int32_t T,
                                              const int32_t* seq_start, int32_t n_seq, float alpha, float* loss,
                                              int32_t* counts, int32_t* seq_counts, int32_t* seq_tokens, void* ws,
                                              size_t ws_bytes, cudaStream_t stream) {
  const flint_moe_status st = check_sizes(c, T, seq_start, n_seq, alpha);
  if (st != FLINT_MOE_OK) return st;
  if (!loss || !counts || !seq_counts || !seq_tokens || !ws || (T > 0 && (!logits || !idx))) return FLINT_MOE_EINVAL;
  if (!aligned(loss, 4) || !aligned(counts, 4) || !aligned(seq_counts, 4) || !aligned(seq_tokens, 4) || !aligned(ws, 16) ||
      !aligned(idx, 4) || !aligned(seq_start, 4) || !aligned(logits, c->num_experts % 4 == 0 ? 16 : 4))
    return FLINT_MOE_EALIGN;
  const BalWs w = bal_ws();
  if (ws_bytes < w.total) return FLINT_MOE_EINVAL;
  BalArgs a = {};
  a.T = T;
  a.E = c->num_experts;
  a.k = c->top_k;
  a.n_seq = n_seq;
  a.alpha = alpha;
  a.logits = logits;
  a.idx = idx;
  a.seq_start = seq_start;
  a.loss = loss;
  a.counts = counts;
  a.seq_counts = seq_counts;
  a.seq_tokens = seq_tokens;
  a.ticket = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(ws) + w.ticket);
  a.partial = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + w.partial);
  k_bal_zero<<<(int)std::min<size_t>(152, ((size_t)n_seq * a.E + 255) / 256), 256, 0, stream>>>(a);
  if (T > 0) {
    k_bal_count<<<std::min(304, (T + 255) / 256), 256, 0, stream>>>(a);
    const int grid = row_blocks(T);
    if (a.E % 4 == 0) {
      if (a.E <= 128) k_bal_loss<4, true><<<grid, 256, 0, stream>>>(a);
      else if (a.E <= 256) k_bal_loss<8, true><<<grid, 256, 0, stream>>>(a);
      else k_bal_loss<16, true><<<grid, 256, 0, stream>>>(a);
    } else {
      k_bal_loss<16, false><<<grid, 256, 0, stream>>>(a);
    }
  }
  return cudaGetLastError() == cudaSuccess ? FLINT_MOE_OK : FLINT_MOE_ECUDA;
}

extern "C" flint_moe_status flint_moe_balance_backward(const flint_moe_config* c, const float* logits, const int32_t* idx,
                                                       int32_t T, const int32_t* seq_start, int32_t n_seq, float alpha,
                                                       const int32_t* seq_counts, const int32_t* seq_tokens,
                                                       const float* dloss, const float* dw, float* dlogits,
                                                       cudaStream_t stream) {
  const flint_moe_status st = check_sizes(c, T, seq_start, n_seq, alpha);
  if (st != FLINT_MOE_OK) return st;
  if (T == 0) return FLINT_MOE_OK;
  if (!logits || !idx || !seq_counts || !seq_tokens || !dlogits) return FLINT_MOE_EINVAL;
  const uintptr_t row = c->num_experts % 4 == 0 ? 16 : 4;
  if (!aligned(logits, row) || !aligned(dlogits, row) || !aligned(idx, 4) || !aligned(seq_start, 4) ||
      !aligned(seq_counts, 4) || !aligned(seq_tokens, 4) || !aligned(dloss, 4) || !aligned(dw, 4))
    return FLINT_MOE_EALIGN;
  const size_t bytes = (size_t)T * c->num_experts * 4;
  if (overlap(logits, bytes, dlogits, bytes)) return FLINT_MOE_EINVAL;
  BalArgs a = {};
  a.T = T;
  a.E = c->num_experts;
  a.k = c->top_k;
  a.n_seq = n_seq;
  a.renorm = c->renormalize;
  a.routed_scale = c->routed_scale;
  a.alpha = alpha;
  a.logits = logits;
  a.idx = idx;
  a.seq_start = seq_start;
  a.seq_counts = const_cast<int32_t*>(seq_counts);
  a.seq_tokens = const_cast<int32_t*>(seq_tokens);
  a.dloss = dloss;
  a.dw = dw;
  a.dlogits = dlogits;
  const int grid = row_blocks(T);
  if (a.E % 4 == 0) {
    if (a.E <= 128) k_bal_backward<4, true><<<grid, 256, 0, stream>>>(a);
    else if (a.E <= 256) k_bal_backward<8, true><<<grid, 256, 0, stream>>>(a);
    else k_bal_backward<16, true><<<grid, 256, 0, stream>>>(a);
  } else {
    k_bal_backward<16, false><<<grid, 256, 0, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? FLINT_MOE_OK : FLINT_MOE_ECUDA;
}
