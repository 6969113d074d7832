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

// Sequence of token t: the last b with seq_start[b] <= t (so an empty sequence is never found), -1 before the
// first, n_seq behind the last. The whole warp searches, 32 places at a time, and gets the same answer: a
// search by halves would wait for one load after another, six of them for 37 sequences.
__device__ __forceinline__ int seq_of(const BalArgs& a, int t, int lane) {
  if (!a.seq_start) return 0;
  int lo = -1, hi = a.n_seq + 1;  // seq_at(lo) <= t < seq_at(hi), taking both ends as given
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step;
    const bool le = i < hi && seq_at(a, i) <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int c = m == 0xffffffffu ? 32 : __ffs(~m) - 1;  // leading lanes that still lie at or before t
    const int nlo = lo + c * step;
    hi = min(hi, nlo + step);
    lo = nlo;
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
  pdl_wait();
  pdl_trigger();
  const size_t n = (size_t)a.n_seq * a.E;
  for (size_t i = blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) a.seq_counts[i] = 0;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < a.n_seq; i += gridDim.x * 256) a.seq_tokens[i] = 0;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < a.E; i += gridDim.x * 256) a.counts[i] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *a.ticket = 0;
    if (a.T == 0) *a.loss = 0.f;
  }
}

// Picks of a block's run of tokens: counted in shared memory, sequence by sequence, and added to the global
// counts once per block and sequence. A piece of a sequence of fewer than SHORT tokens in the run goes to the
// global counts directly: flushing E counters for it would cost more than its own picks do.
constexpr int SHORT = 64;
__global__ void __launch_bounds__(256) k_bal_count(const BalArgs a) {
  __shared__ int hist[MAX_E], total[MAX_E];
  __shared__ int tokens;
  const int lane = threadIdx.x & 31;
  const int per = (a.T + gridDim.x - 1) / gridDim.x;
  const int t0 = min(a.T, (int)blockIdx.x * per), t1 = min(a.T, t0 + per);
  for (int e = threadIdx.x; e < a.E; e += 256) hist[e] = total[e] = 0;
  if (threadIdx.x == 0) tokens = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  if (t0 >= t1) return;
  int b = seq_of(a, t0, lane);
  for (int t = t0; t < t1 && b < a.n_seq;) {  // piece [t, end) of sequence b
    const int end = min(t1, max(t + 1, b < 0 ? seq_at(a, 0) : seq_at(a, b + 1)));
    if (b >= 0) {
      const bool whole = end - t >= SHORT;
      int* sc = a.seq_counts + (size_t)b * a.E;
      int mine = 0;
      for (int i = t + threadIdx.x; i < end; i += 256) {
        const int* p = a.idx + (size_t)i * a.k;
        if (__ldg(p) < 0) continue;
        ++mine;
        for (int j = 0; j < a.k; ++j) {
          const int e = __ldg(p + j);
          if (e < 0 || e >= a.E) continue;
          atomicAdd(total + e, 1);
          if (whole)
            atomicAdd(hist + e, 1);
          else
            atomicAdd(sc + e, 1);
        }
      }
      mine = __reduce_add_sync(0xffffffffu, mine);
      if (whole) {
        if (lane == 0 && mine) atomicAdd(&tokens, mine);
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += 256) {
          if (hist[e]) atomicAdd(sc + e, hist[e]);
          hist[e] = 0;
        }
        if (threadIdx.x == 0) {
          if (tokens) atomicAdd(a.seq_tokens + b, tokens);
          tokens = 0;
        }
        __syncthreads();
      } else if (lane == 0 && mine) {
        atomicAdd(a.seq_tokens + b, mine);
      }
    }
    t = end;
    // the next sequence, or past a run of empty ones the next that holds a token
    b = b + 1 >= a.n_seq || seq_at(a, b + 2) > t ? b + 1 : seq_of(a, t, lane);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += 256)
    if (total[e]) atomicAdd(a.counts + e, total[e]);
}

// The sequence a warp's tokens are in, and that sequence's f - 1 and 1 / T_b.
template <int PER, bool VEC>
struct Cursor {
  int b = -2, end = -1;  // the sequence, and the first token past it
  float inv = 0.f;       // 1 / T_b
  float f[PER];
  __device__ __forceinline__ bool inside(const BalArgs& a) const { return b >= 0 && b < a.n_seq; }
  __device__ __forceinline__ void to(const BalArgs& a, int t, int lane) {
    if (t < end) return;
    b = seq_of(a, t, lane);
    end = max(t + 1, b < 0 ? seq_at(a, 0) : (b < a.n_seq ? seq_at(a, b + 1) : a.T));
    if (inside(a)) {
      const int Tb = __ldcg(a.seq_tokens + b);
      inv = Tb > 0 ? 1.0f / (float)Tb : 0.f;
      load_f<PER, VEC>(a, b, Tb, lane, f);
    }
  }
};

// Consecutive tokens of one warp, so that the warps' runs cover all tokens.
__device__ __forceinline__ void warp_run(const BalArgs& a, int warp, int& t0, int& t1) {
  const int per = (a.T + gridDim.x * 8 - 1) / (gridDim.x * 8);
  t0 = min(a.T, ((int)blockIdx.x * 8 + warp) * per);
  t1 = min(a.T, t0 + per);
}

// Blocks of an SM by registers: a row's values and the next row's take 4 PER of them.
template <int PER>
constexpr int loss_blocks() { return PER > 8 ? 2 : 4; }
template <int PER>
constexpr int backward_blocks() { return PER > 8 ? 1 : 3; }

// Sum over the block's tokens of (1 + F_t) / T_b in FP64; the last block to finish adds the
// blocks' sums in block order. The next token's row is on its way while one is summed up.
template <int PER, bool VEC>
__global__ void __launch_bounds__(256, loss_blocks<PER>()) k_bal_loss(const BalArgs a) {
  __shared__ double red[8];
  __shared__ bool last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int t0, t1;
  warp_run(a, warp, t0, t1);
  float z[PER];
  int first = -1;
  if (t0 < t1) {
    load_row<PER, VEC>(a.logits + (size_t)t0 * a.E, a.E, lane, z);
    first = __ldg(a.idx + (size_t)t0 * a.k);
  }
  pdl_wait();  // the counts
  double acc = 0.0;
  Cursor<PER, VEC> cur;
  for (int t = t0; t < t1; ++t) {
    cur.to(a, t, lane);
    float zn[PER];
    int firstn = -1;
    if (t + 1 < t1) {
      load_row<PER, VEC>(a.logits + (size_t)(t + 1) * a.E, a.E, lane, zn);
      firstn = __ldg(a.idx + (size_t)(t + 1) * a.k);
    }
    if (cur.inside(a) && first >= 0) {
      float s[PER], q[PER];
      const float S = scores<PER, VEC>(z, a.E, lane, s, q);
      float F = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) F = fmaf(cur.f[j], s[j], F);
      F = warp_sum(F);
      // FP32 is enough for one token's share of 1 + F; the long sum is held in FP64
      if (S > 0.f) acc += (double)((1.0f + F / S) * cur.inv);
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) z[j] = zn[j];
    first = firstn;
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
__global__ void __launch_bounds__(256, backward_blocks<PER>()) k_bal_backward(const BalArgs a) {
  __shared__ float extra_s[8][MAX_E];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int t0, t1;
  warp_run(a, warp, t0, t1);
  float* extra = extra_s[warp];  // routing-weight part of the row's gradient, zero but at its picks
  for (int e = lane; e < a.E; e += 32) extra[e] = 0.f;
  pdl_wait();
  pdl_trigger();
  __syncwarp();
  const float up = (a.dloss ? __ldg(a.dloss) : 1.0f) * (a.alpha / (float)a.n_seq);
  const bool mine = lane < a.k;
  float z[PER];
  int e = -1;
  float g = 0.f;
  if (t0 < t1) {
    load_row<PER, VEC>(a.logits + (size_t)t0 * a.E, a.E, lane, z);
    if (mine) e = __ldg(a.idx + (size_t)t0 * a.k + lane);
    if (mine && a.dw) g = __ldg(a.dw + (size_t)t0 * a.k + lane);
  }
  Cursor<PER, VEC> cur;
  for (int t = t0; t < t1; ++t) {
    cur.to(a, t, lane);
    float zn[PER];
    int en = -1;
    float gn = 0.f;
    if (t + 1 < t1) {  // the next token's row is on its way while this one is worked on
      load_row<PER, VEC>(a.logits + (size_t)(t + 1) * a.E, a.E, lane, zn);
      if (mine) en = __ldg(a.idx + (size_t)(t + 1) * a.k + lane);
      if (mine && a.dw) gn = __ldg(a.dw + (size_t)(t + 1) * a.k + lane);
    }
    if (cur.inside(a)) {
      const float* row = a.logits + (size_t)t * a.E;
      float* out = a.dlogits + (size_t)t * a.E;
      const bool counted = __shfl_sync(0xffffffffu, e, 0) >= 0;
      float d[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) d[j] = 0.f;
      if (counted) {
        float s[PER], q[PER];
        const float S = scores<PER, VEC>(z, a.E, lane, s, q);
        float F = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) F = fmaf(cur.f[j], s[j], F);
        F = warp_sum(F);
        const float inv = S > 0.f ? 1.0f / S : 0.f;
        F *= inv;
        const float ci = up * cur.inv * inv;
#pragma unroll
        for (int j = 0; j < PER; ++j) d[j] = (ci * s[j]) * ((cur.f[j] - F) * q[j]);
        if (a.dw) {
          const bool in = e >= 0 && e < a.E;
          float sp = 0.f, qp = 0.f, zp = -INFINITY;
          if (in) {
            zp = __ldg(row + e);
            sigmoid2(zp, sp, qp);
          }
          float add;
          if (a.renorm) {
            float W = warp_sum(sp);
            if (W < LOW_ROW * MAX_TOPK) {  // every pick's score underflows: the same shares from exp(z - max z)
              const float m = warp_max(zp);
              sp = in && m > -INFINITY ? __expf(zp - m) : 0.f;
              W = warp_sum(sp);
            }
            const float w = W > 0.f ? sp / W : 0.f;
            const float D = warp_sum(in ? g * w : 0.f);
            add = in ? a.routed_scale * w * (g - D) * qp : 0.f;
          } else {
            add = in ? a.routed_scale * sp * g * qp : 0.f;
          }
          // An expert picked twice: the picks' parts are added in pick order. Each pick signs its expert's
          // place, and finds another's name there if it is not alone (a match over 32 different values
          // took longer than the rest of the row: 67 us for 65536 x 256, of 41 million instructions).
          if (in) reinterpret_cast<int*>(extra)[e] = lane;
          __syncwarp();
          const bool shared = in && reinterpret_cast<const int*>(extra)[e] != lane;
          float sum = add;
          if (__any_sync(0xffffffffu, shared)) {
            sum = 0.f;
            for (int j = 0; j < a.k; ++j) {
              const float v = __shfl_sync(0xffffffffu, add, j);
              if (__shfl_sync(0xffffffffu, e, j) == e) sum += v;
            }
          }
          __syncwarp();
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
          const int el = 4 * (lane + 32 * i);
          if (el < a.E)
            *reinterpret_cast<float4*>(out + el) = make_float4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < PER; ++j)
          if (lane + 32 * j < a.E) out[lane + 32 * j] = d[j];
      }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) z[j] = zn[j];
    e = en;
    g = gn;
  }
}

}  // namespace bal
}  // namespace flint

using namespace flint;
using namespace flint::bal;

namespace {

constexpr int SMS = 152;
constexpr int LOSS_BLOCKS = SMS * loss_blocks<4>();  // the loss kernel's blocks at most
constexpr int COUNT_BLOCKS = SMS;

// A launch that may start while the kernel before it drains (each kernel waits for it itself).
bool launch(void (*kernel)(BalArgs), int grid, cudaStream_t stream, const BalArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess;
}

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

// One warp per token while tokens are few, then as many blocks as run at once.
int row_blocks(int T, int per_sm) { return std::min((T + 7) / 8, SMS * per_sm); }

template <int PER, bool VEC>
bool launch_loss(const BalArgs& a, cudaStream_t stream) {
  return launch(k_bal_loss<PER, VEC>, row_blocks(a.T, loss_blocks<PER>()), stream, a);
}
template <int PER, bool VEC>
bool launch_backward(const BalArgs& a, cudaStream_t stream) {
  return launch(k_bal_backward<PER, VEC>, row_blocks(a.T, backward_blocks<PER>()), stream, a);
}

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
  bool ok = launch(k_bal_zero, (int)std::min<size_t>(152, ((size_t)n_seq * a.E + 255) / 256), stream, a);
  if (T > 0) {
    ok = ok && launch(k_bal_count, std::min(COUNT_BLOCKS, (T + 255) / 256), stream, a);
    ok = ok && (a.E % 4 != 0 ? launch_loss<16, false>(a, stream)
                : a.E <= 128 ? launch_loss<4, true>(a, stream)
                : a.E <= 256 ? launch_loss<8, true>(a, stream)
                             : launch_loss<16, true>(a, stream));
  }
  return ok ? FLINT_MOE_OK : FLINT_MOE_ECUDA;
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
  const bool ok = a.E % 4 != 0 ? launch_backward<16, false>(a, stream)
                  : a.E <= 128 ? launch_backward<4, true>(a, stream)
                  : a.E <= 256 ? launch_backward<8, true>(a, stream)
                               : launch_backward<16, true>(a, stream);
  return ok ? FLINT_MOE_OK : FLINT_MOE_ECUDA;
}
