// Balance loss of the router with per-expert counts, and the gradient of the
// router's logits (C ABI: include/flint_moe_balance.h).
//
// One pass over the logits each way. With f_be - 1 = (E c_be - k T_b) / (k T_b)
// (whole numbers until the division, so nothing cancels) and sum_e p_te = 1,
//   sum_e f_be p_te = 1 + F_t,   F_t = sum_e (f_be - 1) s_te / sum_e s_te
//   loss = alpha / n_seq  sum_t (1 + F_t) / T_b
//   dz_tj = dloss alpha / (n_seq T_b) p_tj ((f_bj - 1) - F_t) (1 - s_tj)
// so a row of the gradient needs two sums, sum_e s and sum_e (f - 1) s, and no
// second look at memory, and the loss, summed over tokens first, sum_e s only
// (k_bal_loss). The counts come from the picks alone.
//
// One warp per token row, 16-byte copies. The rows are bound by memory bandwidth
// and nearly as much by instructions; the counts by latency.
// 65536 tokens of 256 experts, alone and cold: zeros 2.2 us, counts 8.4, loss 23.8
// (69 MB), gradient 29.9 (67 MB in, 67 MB out: 4.5 TB/s); whole calls 28.0 and 32.0.
#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "flint_moe_balance.h"

namespace flint {
namespace bal {

constexpr int MAX_E = MAX_EXPERTS;

struct BalArgs {
  int T, E, k, n_seq, renorm;
  bool narrow;  // k T E < 2^31
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

// The hardware's exponential and reciprocal with subnormal results flushed: none occur below, and the rows are
// bound by instructions otherwise (the forms that keep them take three times as many).
__device__ __forceinline__ float exp_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float rcp_of(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The smaller of both, NaN if one is: a NaN logit must not look like a very negative one.
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// s = sigmoid(z) and q = 1 - s without cancellation: with e = exp(-z), s = 1 / (1 + e) and
// q = e s. Scores below the smallest FP32 normal (z under -87.3) are zero, and e is held
// below infinity in q only, so that e s s is zero there. Rows in which no s is above 1e-12
// take the shares of exp(z - max z) instead, which are theirs to 1e-12 E < 2^-30 of the
// value (sigmoid(z) = exp(z) / (1 + exp(z))): so what is lost to zero is below 1e-26 of a row.
constexpr float LOW_ROW = 1e-12f;
constexpr float E_MOST = 8.5e37f;  // 2^126: 1 / (1 + e) of a larger e is zero
__device__ __forceinline__ void sigmoid2(float z, float& s, float& q) {
  const float e = exp_of(-z);
  s = rcp_of(1.0f + e);
  q = e > 1e9f ? 1.0f : e * s;
}

// Pairs of FP32 values in one instruction.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float ex2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's logits: lane l holds elements 4 (l + 32 i) .. + 3 (VEC, E % 4 == 0) or l + 32 i.
template <bool VEC>
__device__ __forceinline__ int elem(int lane, int j) {
  return VEC ? 4 * (lane + 32 * (j >> 2)) + (j & 3) : lane + 32 * j;
}

// -infinity stands for the places past E: their s is zero.
template <int PER, bool VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float (&z)[PER]) {
  if (VEC) {
#pragma unroll
    for (int i = 0; i < PER / 4; ++i) {
      const int e = 4 * (lane + 32 * i);
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) v = __ldg(reinterpret_cast<const float4*>(row + e));
      z[4 * i] = v.x;
      z[4 * i + 1] = v.y;
      z[4 * i + 2] = v.z;
      z[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) z[j] = lane + 32 * j < E ? __ldg(row + lane + 32 * j) : -INFINITY;
  }
}

// Sums of a row: this lane's parts of sum s and sum f s. exp(-z) may overflow to infinity here: that s is 0.
template <int PER>
__device__ __forceinline__ void row_sums(const float (&z)[PER], const float (&f)[PER], float& S, float& F) {
  f32x2 S2 = 0ull, F2 = 0ull;  // two zeros each
  const f32x2 one = pack2(1.f, 1.f), k = pack2(-LOG2E, -LOG2E);
#pragma unroll
  for (int j = 0; j < PER; j += 2) {
    float a, b;
    unpack2(mul2(pack2(z[j], z[j + 1]), k), a, b);
    unpack2(add2(pack2(ex2_of(a), ex2_of(b)), one), a, b);
    const f32x2 s = pack2(rcp_of(a), rcp_of(b));
    S2 = add2(S2, s);
    F2 = fma2(pack2(f[j], f[j + 1]), s, F2);
  }
  float a, b;
  unpack2(S2, a, b);
  S = a + b;
  unpack2(F2, a, b);
  F = a + b;
}

// A low row: no s above LOW_ROW, the shares from exp(z - max z) instead. s: this lane's of them (0 for a row of
// -infinity), S and F the row's sums.
template <int PER>
__device__ __noinline__ void low_row(const float (&z)[PER], const float (&f)[PER], float (&s)[PER], float& S, float& F) {
  float m = z[0];
#pragma unroll
  for (int j = 1; j < PER; ++j) m = fmaxf(m, z[j]);
  m = warp_max(m);
  S = F = 0.f;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    s[j] = m > -INFINITY ? exp_of(z[j] - m) : 0.f;
    S += s[j];
    F = fmaf(f[j], s[j], F);
  }
  S = warp_sum(S);
  F = warp_sum(F);
}

// One step of sums over lanes of 2 N values at once: the lanes whose `bit` is set go on with the upper N, the others
// with the lower N, each having got the other lanes' share of them.
template <int N>
__device__ __forceinline__ void halve(float (&v)[2 * N], int lane, int bit) {
  const bool up = lane & bit;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float keep = up ? v[j + N] : v[j], send = up ? v[j] : v[j + N];
    v[j] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
  }
}
template <int N>
__device__ __forceinline__ float (&first_of(float (&v)[2 * N]))[N] { return reinterpret_cast<float (&)[N]>(v); }

// f - 1 of an expert with c of a sequence's picks, even = k T_b and inv = 1 / even (0 for none). The difference is a
// whole number; `narrow`: it fits 32 bits (k T E does), and its conversion spares the FP64 unit.
__device__ __forceinline__ float load_of(int c, int E, int even, float inv, bool narrow) {
  return (narrow ? (float)(c * E - even) : (float)((long long)c * E - even)) * inv;
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
// counts once per block and sequence. A piece of a sequence of fewer than SHORT tokens goes to the global counts
// directly: flushing E counters for it would cost more than its own picks do. The picks, one run of memory, come to
// shared memory up to COUNT_INTS at a time, all asked for at once.
constexpr int SHORT = 64;
constexpr int COUNT_INTS = 2048;
__global__ void __launch_bounds__(256) k_bal_count(const BalArgs a) {
  __shared__ int hist[MAX_E], total[MAX_E], picks[COUNT_INTS];
  __shared__ int tokens;
  const int lane = threadIdx.x & 31;
  const int per = (a.T + gridDim.x - 1) / gridDim.x;
  const int t0 = min(a.T, (int)blockIdx.x * per), t1 = min(a.T, t0 + per);
  for (int e = threadIdx.x; e < a.E; e += 256) hist[e] = total[e] = 0;
  if (threadIdx.x == 0) tokens = 0;
  pdl_trigger();  // the rows' kernel needs what is written here at its end only
  pdl_wait();
  if (t0 >= t1) return;
  int b = seq_of(a, t0, lane);
  for (int t = t0; t < t1 && b < a.n_seq;) {  // piece [t, end) of sequence b
    const int end = min(min(t1, t + COUNT_INTS / a.k), max(t + 1, seq_at(a, b + 1)));
    if (b >= 0) {
      const bool whole = end - t >= SHORT;
      int* sc = a.seq_counts + (size_t)b * a.E;
      const int n = (end - t) * a.k;
      __syncthreads();  // the picks before have been counted
#pragma unroll 4
      for (int i = threadIdx.x; i < n; i += 256) picks[i] = __ldg(a.idx + (size_t)t * a.k + i);
      __syncthreads();
      int mine = 0;
#pragma unroll 1
      for (int i = threadIdx.x; i < n; i += 256) {
        const int at = i / a.k * a.k, e = picks[i];  // a token's first pick tells whether it counts
        if (picks[at] < 0) continue;
        if (at == i) ++mine;
        if (e < 0 || e >= a.E) continue;
        atomicAdd(total + e, 1);
        atomicAdd(whole ? hist + e : sc + e, 1);
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
      } else if (lane == 0 && mine) {
        atomicAdd(a.seq_tokens + b, mine);
      }
    }
    t = end;
    // still this sequence (or before the first, whose pieces end before its start too), the next one, or past a run of
    // empty ones the next that holds a token
    if (seq_at(a, b + 1) <= t) b = b + 1 >= a.n_seq || seq_at(a, b + 2) > t ? b + 1 : seq_of(a, t, lane);
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
  // The sequence of token t, without its counts.
  __device__ __forceinline__ void find(const BalArgs& a, int t, int lane) {
    b = seq_of(a, t, lane);
    end = max(t + 1, b < 0 ? seq_at(a, 0) : (b < a.n_seq ? seq_at(a, b + 1) : a.T));
  }
  __device__ __forceinline__ void to(const BalArgs& a, int t, int lane) {
    if (t < end) return;
    find(a, t, lane);
    load(a, lane);
  }
  __device__ __forceinline__ void load(const BalArgs& a, int lane) {
    int raw[PER], Tb = 0;
    ask(a, lane, raw, Tb);
    settle(a, lane, raw, Tb);
  }
  // The counts' loads, and what follows from them.
  __device__ __forceinline__ void ask(const BalArgs& a, int lane, int (&raw)[PER], int& Tb) const {
    Tb = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) raw[j] = 0;
    if (inside(a)) {
      const int* c = a.seq_counts + (size_t)b * a.E;
      Tb = __ldcg(a.seq_tokens + b);
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int e = elem<VEC>(lane, j);
        if (e < a.E) raw[j] = __ldcg(c + e);
      }
    }
  }
  __device__ __forceinline__ void settle(const BalArgs& a, int lane, const int (&raw)[PER], int Tb) {
    const int even = a.k * Tb;
    const float inv_even = Tb > 0 ? 1.0f / (float)even : 0.f;
    inv = Tb > 0 ? 1.0f / (float)Tb : 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) f[j] = elem<VEC>(lane, j) < a.E ? load_of(raw[j], a.E, even, inv_even, a.narrow) : 0.f;
  }
};

// Consecutive tokens of one warp, so that the warps' runs cover all tokens.
__device__ __forceinline__ void warp_run(const BalArgs& a, int warp, int& t0, int& t1) {
  const int per = (a.T + gridDim.x * 8 - 1) / (gridDim.x * 8);
  t0 = min(a.T, ((int)blockIdx.x * 8 + warp) * per);
  t1 = min(a.T, t0 + per);
}

// Blocks of an SM, by registers (a row's values take four to five times PER) and by the rows in flight.
template <int PER>
constexpr int loss_blocks() { return PER > 8 ? 2 : PER > 4 ? 3 : 4; }
template <int PER>
constexpr int backward_blocks() { return PER > 8 ? 2 : 3; }

// Rows on their way: each lane copies what it will read itself of the next DEPTH rows into shared memory, so nobody
// waits for anybody, and a warp has DEPTH rows in flight where registers hold one or two (2.8 TB/s).
template <int PER, bool VEC>
struct RowRing {
  static constexpr int DEPTH = PER > 8 ? 4 : 8;
  static constexpr int ROW = PER * 32;  // floats of a slot
  float* slots;                         // this warp's
  const float* base;                    // row 0 of the matrix
  int E, next, end, lane;
  __device__ __forceinline__ void issue() {
    if (next < end) {
      float* s = slots + (next & (DEPTH - 1)) * ROW;
      const float* row = base + (size_t)next * E;
      if (VEC) {
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
          const int e = 4 * (lane + 32 * i);
          if (e < E)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(s + e)), "l"(row + e) : "memory");
        }
      } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int e = lane + 32 * j;
          if (e < E) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(s + e)), "l"(row + e) : "memory");
        }
      }
      ++next;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ RowRing(float* smem, const float* logits, int E_, int t0, int t1, int warp, int lane_)
      : slots(smem + warp * DEPTH * ROW), base(logits), E(E_), next(t0), end(t1), lane(lane_) {
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) issue();
  }
  // Row t (in order, each once), and the copy of one more row behind the last.
  __device__ __forceinline__ void take(int t, float (&z)[PER]) {
    issue();
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    const float* s = slots + (t & (DEPTH - 1)) * ROW;
    if (VEC) {
#pragma unroll
      for (int i = 0; i < PER / 4; ++i) {
        const int e = 4 * (lane + 32 * i);
        uint4 v = make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);  // -infinity past E
        if (e < E) v = lds128(s + e);
        z[4 * i] = __uint_as_float(v.x);
        z[4 * i + 1] = __uint_as_float(v.y);
        z[4 * i + 2] = __uint_as_float(v.z);
        z[4 * i + 3] = __uint_as_float(v.w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) z[j] = lane + 32 * j < E ? __uint_as_float(lds32(s + lane + 32 * j)) : -INFINITY;
    }
  }
  static size_t bytes() { return sizeof(float) * 8 * DEPTH * ROW; }
};

// The loss is sum_b 1/T_b (tokens + sum_e (f_be - 1) P_be) with P_be = sum_t p_te, so the rows need no counts: a warp
// adds up its tokens' shares in registers, expert by expert, beside the kernels that count, and multiplies them by f - 1
// at the end of its piece of a sequence (with the counts first and f in every row: 28.6 us for 65536 x 256). Shares are
// summed in FP32 16 tokens at a time and those sums in FP32 again, everything behind that in FP64; the last block to
// finish adds the blocks' sums, in a fixed order.
template <int PER, bool VEC>
__global__ void __launch_bounds__(256, loss_blocks<PER>()) k_bal_loss(const BalArgs a) {
  extern __shared__ __align__(16) float ring_smem[];
  __shared__ double red[8];
  __shared__ bool last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int t0, t1;
  warp_run(a, warp, t0, t1);
  RowRing<PER, VEC> rows(ring_smem, a.logits, a.E, t0, t1, warp, lane);
  Cursor<PER, VEC> cur;
  float P[PER], Q[PER];  // shares of up to 16 tokens, and of those before
  int counted = 0, n = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) P[j] = Q[j] = 0.f;
  double acc = 0.0;
  for (int t = t0; t < t1;) {
    if (t >= cur.end) cur.find(a, t, lane);
    const int nb = min(2, min(t1, cur.end) - t);  // tokens of one sequence
    // bit r: token t + r counts
    const unsigned live = cur.inside(a) ? __ballot_sync(0xffffffffu, lane < nb && __ldg(a.idx + (size_t)(t + lane) * a.k) >= 0) : 0u;
    f32x2 sv[2][PER / 2];
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (r >= nb) break;
      float z[PER];
      rows.take(t + r, z);
      f32x2 S2 = 0ull;
      const f32x2 one = pack2(1.f, 1.f), k = pack2(-LOG2E, -LOG2E);
#pragma unroll
      for (int j = 0; j < PER; j += 2) {  // exp(-z) may overflow to infinity here: that s is 0
        float x, y;
        unpack2(mul2(pack2(z[j], z[j + 1]), k), x, y);
        unpack2(add2(pack2(ex2_of(x), ex2_of(y)), one), x, y);
        sv[r][j / 2] = pack2(rcp_of(x), rcp_of(y));
        S2 = add2(S2, sv[r][j / 2]);
      }
      float x, y;
      unpack2(S2, x, y);
      v[r] = x + y;
    }
    halve<1>(v, lane, 16);
    float x = v[0];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float S = __shfl_sync(0xffffffffu, x, 16 * r);
      if (!((live >> r) & 1u)) continue;
      if (S < LOW_ROW * a.E) {  // rare: the row again
        float z[PER], s[PER], zero[PER], F;
        load_row<PER, VEC>(a.logits + (size_t)(t + r) * a.E, a.E, lane, z);
#pragma unroll
        for (int j = 0; j < PER; ++j) zero[j] = 0.f;
        low_row<PER>(z, zero, s, S, F);
#pragma unroll
        for (int j = 0; j < PER; j += 2) sv[r][j / 2] = pack2(s[j], s[j + 1]);
      }
      if (S == 0.f) continue;  // a row of -infinity has no shares
      ++counted;
      const float inv = rcp_of(S);
#pragma unroll
      for (int j = 0; j < PER; j += 2) unpack2(fma2(sv[r][j / 2], pack2(inv, inv), pack2(P[j], P[j + 1])), P[j], P[j + 1]);
    }
    t += nb;
    const bool flush = t >= t1 || t >= cur.end;
    if (flush || ++n == 8) {
      n = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        Q[j] += P[j];
        P[j] = 0.f;
      }
    }
    if (flush && counted) {
      pdl_wait();  // the counts
      cur.load(a, lane);
      float d = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) d = fmaf(cur.f[j], Q[j], d);
      acc += ((double)d + (lane == 0 ? (double)counted : 0.0)) * (double)cur.inv;
    }
    if (flush) {
      counted = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) Q[j] = 0.f;
    }
  }
  pdl_wait();  // (also of warps without tokens: the ticket)
  acc = warp_sum_d(acc);
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
  if (!last) return;
  // the blocks' sums: one load or two a thread (by one warp, fifteen in a row, this took a third of the kernel)
  __threadfence();
  double v = 0.0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += 256) v += __ldcg(a.partial + i);
  v = warp_sum_d(v);
  __syncthreads();  // red[] has been read
  if (lane == 0) red[warp] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    double sum = 0.0;
    for (int w = 0; w < 8; ++w) sum += red[w];
    *a.loss = (float)(sum * ((double)a.alpha / (double)a.n_seq));
  }
}

// Counts and loss of a small call in one block: the counts stay in shared memory, and one launch replaces three.
// Its rule (one_block below) is where one SM's share of the work takes no longer than the launches it saves: 300 x 16
// takes 15 us in three kernels.
constexpr int ONE_COUNTS = 8192, ONE_ELEMS = 65536, ONE_TOKENS = 1024;
template <int PER, bool VEC>
__global__ void __launch_bounds__(1024) k_bal_one(const BalArgs g) {
  constexpr int AT = PER > 8 ? 1 : 4;  // rows of a warp in flight
  __shared__ int counts[ONE_COUNTS], tokens[ONE_TOKENS], starts[ONE_TOKENS + 1], seq[ONE_TOKENS];
  __shared__ double red[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < g.n_seq * g.E; i += 1024) counts[i] = 0;
  for (int i = threadIdx.x; i < g.n_seq; i += 1024) tokens[i] = 0;
  pdl_wait();
  pdl_trigger();
  const int t = threadIdx.x;  // this thread's token
  int first = -1;
  if (t < g.T) first = __ldg(g.idx + (size_t)t * g.k);
  for (int i = threadIdx.x; i <= g.n_seq; i += 1024) starts[i] = seq_at(g, i);
  __syncthreads();
  if (t < g.T) {
    int lo = -1, hi = g.n_seq + 1;  // the last sequence that starts at or before t
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (starts[m] <= t)
        lo = m;
      else
        hi = m;
    }
    const bool counted = lo >= 0 && lo < g.n_seq && first >= 0;
    seq[t] = counted ? lo : -1;
    if (counted) {
      atomicAdd(tokens + lo, 1);
      for (int j = 0; j < g.k; ++j) {
        const int e = j ? __ldg(g.idx + (size_t)t * g.k + j) : first;
        if (e >= 0 && e < g.E) atomicAdd(counts + lo * g.E + e, 1);
      }
    }
  }
  const int per = (g.T + 31) / 32, t0 = min(g.T, warp * per), t1 = min(g.T, t0 + per);
  float z[AT][PER];
#pragma unroll
  for (int i = 0; i < AT; ++i)
    if (t0 + i < t1) load_row<PER, VEC>(g.logits + (size_t)(t0 + i) * g.E, g.E, lane, z[i]);
  __syncthreads();
  for (int i = threadIdx.x; i < g.n_seq * g.E; i += 1024) g.seq_counts[i] = counts[i];
  for (int i = threadIdx.x; i < g.n_seq; i += 1024) g.seq_tokens[i] = tokens[i];
  for (int e = threadIdx.x; e < g.E; e += 1024) {
    int c = 0;
    for (int b = 0; b < g.n_seq; ++b) c += counts[b * g.E + e];
    g.counts[e] = c;
  }
  int b = -1;
  float f[PER], inv = 0.f;
  double acc = 0.0;
  for (int i0 = t0; i0 < t1; i0 += AT) {
#pragma unroll
    for (int i = 0; i < AT; ++i) {
      if (i0 + i >= t1) break;
      const int own = seq[i0 + i];
      if (own >= 0 && own != b) {
        b = own;
        const int even = g.k * tokens[b];
        inv = 1.0f / (float)tokens[b];
        const float inv_even = 1.0f / (float)even;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int e = elem<VEC>(lane, j);
          f[j] = e < g.E ? load_of(counts[b * g.E + e], g.E, even, inv_even, true) : 0.f;
        }
      }
      if (own >= 0) {
        float S, F;
        row_sums<PER>(z[i], f, S, F);
        S = warp_sum(S);
        F = warp_sum(F);
        if (S < LOW_ROW * g.E) {
          float s[PER];
          low_row<PER>(z[i], f, s, S, F);
        }
        if (S != 0.f) acc += (double)((1.0f + __fdividef(F, S)) * inv);
      }
      if (i0 + AT + i < t1) load_row<PER, VEC>(g.logits + (size_t)(i0 + AT + i) * g.E, g.E, lane, z[i]);
    }
  }
  if (lane == 0) red[warp] = acc;
  __syncthreads();
  if (warp == 0) {
    const double v = warp_sum_d(red[lane]);
    if (lane == 0) *g.loss = (float)(v * ((double)g.alpha / (double)g.n_seq));
  }
}

// A warp works on NB tokens at a time: their rows for the loss's part, then the
// NB tokens' picks side by side, 32 / NB lanes to a token (k <= 8: four tokens; picks of one token at a time would
// leave three lanes in four idle, and the kernel is bound by instructions before it is bound by memory). A pick
// adds its part to its place in the row just written.
template <int PER, bool VEC, int NB>
__global__ void __launch_bounds__(256, backward_blocks<PER>()) k_bal_backward(const BalArgs a) {
  extern __shared__ __align__(16) float ring_smem[];
  constexpr int W = 32 / NB;  // lanes of a token's picks
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = lane / W, pick = lane % W;
  int t0, t1;
  warp_run(a, warp, t0, t1);
  pdl_wait();
  pdl_trigger();
  const float up = (a.dloss ? __ldg(a.dloss) : 1.0f) * (a.alpha / (float)a.n_seq);
  // The first sequence's counts are asked for before the rows, behind which they would wait for microseconds.
  Cursor<PER, VEC> cur;
  int raw[PER], Tb = 0;
  if (t0 < t1) cur.find(a, t0, lane);
  cur.ask(a, lane, raw, Tb);
  RowRing<PER, VEC> rows(ring_smem, a.logits, a.E, t0, t1, warp, lane);
  cur.settle(a, lane, raw, Tb);
  // This lane's pick of token t + slot, and its gradient, asked for a step ahead, as they wait behind the rows in flight
  // (65536 x 256: 32.8 -> 32.0 us).
  auto pick_of = [&](int t) { return t + slot < t1 && pick < a.k ? __ldg(a.idx + (size_t)(t + slot) * a.k + pick) : -1; };
  auto grad_of = [&](int t) { return a.dw && t + slot < t1 && pick < a.k ? __ldg(a.dw + (size_t)(t + slot) * a.k + pick) : 0.f; };
  int e_next = pick_of(t0);
  float g_next = grad_of(t0);
  for (int t = t0; t < t1;) {
    cur.to(a, t, lane);
    const int nb = min(NB, min(t1, cur.end) - t);  // tokens of one sequence
    const int e = slot < nb ? e_next : -1;
    const float g_here = g_next;
    e_next = pick_of(t + nb);
    g_next = grad_of(t + nb);
    const unsigned pads = __ballot_sync(0xffffffffu, pick == 0 && e < 0);  // bit W i: token i is padding
    const bool in = e >= 0 && e < a.E && !((pads >> (slot * W)) & 1u) && cur.inside(a);
    float g = 0.f, zp = -INFINITY;
    if (a.dw && in) {
      g = g_here;
      zp = __ldg(a.logits + (size_t)(t + slot) * a.E + e);
    }
    // Two rows at a time: their four sums over the lanes at once.
#pragma unroll 1
    for (int i = 0; i < nb; i += 2) {
      f32x2 sq[2][PER / 2];  // s (1 - s)
      float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (i + r >= nb) break;
        float z[PER];
        rows.take(t + i + r, z);
        f32x2 S2 = 0ull, F2 = 0ull;
        const f32x2 one = pack2(1.f, 1.f), k = pack2(-LOG2E, -LOG2E);
#pragma unroll
        for (int j = 0; j < PER; j += 2) {
          float x, y;
          unpack2(mul2(pack2(z[j], z[j + 1]), k), x, y);
          x = ex2_of(x);
          y = ex2_of(y);
          const f32x2 e = pack2(min_nan(x, E_MOST), min_nan(y, E_MOST));  // so that e s is no infinity times 0
          unpack2(add2(pack2(x, y), one), x, y);
          const f32x2 s = pack2(rcp_of(x), rcp_of(y));
          S2 = add2(S2, s);
          F2 = fma2(pack2(cur.f[j], cur.f[j + 1]), s, F2);
          sq[r][j / 2] = mul2(mul2(e, s), s);
        }
        float x, y;
        unpack2(S2, x, y);
        v[r] = x + y;
        unpack2(F2, x, y);
        v[2 + r] = x + y;
      }
      halve<2>(v, lane, 16);
      halve<1>(first_of<2>(v), lane, 8);
      float x = v[0];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      if (!cur.inside(a)) continue;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (i + r >= nb) break;
        float S = __shfl_sync(0xffffffffu, x, 8 * r), F = __shfl_sync(0xffffffffu, x, 16 + 8 * r);
        float* out = a.dlogits + (size_t)(t + i + r) * a.E;
        const bool pad = (pads >> ((i + r) * W)) & 1u;  // a padding row may hold anything: it is not multiplied
        if (!pad && S < LOW_ROW * a.E) {
          float z[PER], s[PER];
          load_row<PER, VEC>(a.logits + (size_t)(t + i + r) * a.E, a.E, lane, z);
          low_row<PER>(z, cur.f, s, S, F);
#pragma unroll
          for (int j = 0; j < PER; j += 2) {
            float s0, q0, s1, q1;
            sigmoid2(z[j], s0, q0);
            sigmoid2(z[j + 1], s1, q1);
            sq[r][j / 2] = pack2(s[j] * q0, s[j + 1] * q1);
          }
        }
        const float inv = S != 0.f ? rcp_of(S) : 0.f, ci = up * cur.inv * inv, off = -F * inv * ci;
        float d[PER];
#pragma unroll
        for (int j = 0; j < PER; j += 2)
          unpack2(mul2(sq[r][j / 2], fma2(pack2(cur.f[j], cur.f[j + 1]), pack2(ci, ci), pack2(off, off))), d[j], d[j + 1]);
        if (pad) {
#pragma unroll
          for (int j = 0; j < PER; ++j) d[j] = 0.f;
        }
        if (VEC) {
#pragma unroll
          for (int j = 0; j < PER / 4; ++j) {
            const int el = 4 * (lane + 32 * j);
            if (el < a.E)
              *reinterpret_cast<float4*>(out + el) = make_float4(d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < PER; ++j)
            if (lane + 32 * j < a.E) out[lane + 32 * j] = d[j];
        }
      }
    }
    if (a.dw && cur.inside(a)) {
      // sums over a token's lanes
      auto sum_of = [&](float v) {
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
      };
      float sp = 0.f, qp = 0.f;
      if (in) sigmoid2(zp, sp, qp);
      float add = sp * g * qp;
      if (a.renorm) {
        float total = sum_of(sp);
        if (__any_sync(0xffffffffu, total < LOW_ROW * MAX_TOPK)) {
          // every score of a token's picks underflows: the same shares from exp(z - max z)
          float m = zp;
#pragma unroll
          for (int o = W / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (total < LOW_ROW * MAX_TOPK) sp = in && m > -INFINITY ? exp_of(zp - m) : 0.f;
          total = sum_of(sp);
        }
        // The weights' sum of one makes any constant in g drop out: a token of one pick gets an exact zero, whatever the
        // quotient's rounding (and NaN shows). Of several picks nothing is taken off: where a pick of a small weight has
        // a large g, the others would lose their digits.
        const unsigned ins = __ballot_sync(0xffffffffu, in) >> (slot * W) & ((1u << W) - 1);
        if (__popc(ins) == 1) g -= g;
        const float w = total != 0.f ? __fdividef(sp, total) : 0.f;
        add = w * (g - sum_of(g * w)) * qp;
      }
      add *= a.routed_scale;
      // An expert picked twice gets its picks' parts in pick order; each of them writes the same value.
      float part = 0.f;
      for (int j = 0; j < a.k; ++j) {
        const int ej = __shfl_sync(0xffffffffu, e, slot * W + j);
        const float v = __shfl_sync(0xffffffffu, add, slot * W + j);
        if (ej == e) part += v;
      }
      __syncwarp();  // the rows are written
      float* place = a.dlogits + (size_t)(t + slot) * a.E + e;
      float base = 0.f;
      if (in) base = *place;
      __syncwarp();
      if (in) *place = base + part;
    }
    t += nb;
  }
}

}  // namespace bal
}  // namespace flint

using namespace flint;
using namespace flint::bal;

namespace {

constexpr int SMS = 152;
constexpr int LOSS_BLOCKS = SMS * 4;  // the loss kernel's blocks at most
constexpr int COUNT_BLOCKS = 2 * SMS;

// Prepares a kernel once for each device: its dynamic shared memory, and the largest shared-memory carveout, which all
// kernels of a call ask for, because an SM runs blocks of two kernels side by side only under one carveout.
bool prepare(void (*kernel)(BalArgs), std::atomic<uint64_t>& done, size_t smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev > 63) return false;
  if ((done.load() >> dev) & 1) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared) !=
          cudaSuccess ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return false;
  done.fetch_or((uint64_t)1 << dev);
  return true;
}

// A launch that may start while the kernel before it drains (each kernel waits for it itself).
bool launch(void (*kernel)(BalArgs), int grid, cudaStream_t stream, const BalArgs& a, int block = 256, size_t smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
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

struct Span {
  const void* p;
  size_t n;
};
// Whether one of the outputs shares memory with another or with an input: kernels of a call write the one while they
// read or add to the other.
bool overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  auto meet = [](const Span& u, const Span& v) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(u.p), b = reinterpret_cast<uintptr_t>(v.p);
    return u.p && v.p && u.n && v.n && a < b + v.n && b < a + u.n;
  };
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (meet(*o, *q)) return true;
    for (const Span& i : ins)
      if (meet(*o, i)) return true;
  }
  return false;
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
  static std::atomic<uint64_t> done{0};
  const size_t smem = RowRing<PER, VEC>::bytes();
  return prepare(k_bal_loss<PER, VEC>, done, smem) &&
         launch(k_bal_loss<PER, VEC>, row_blocks(a.T, loss_blocks<PER>()), stream, a, 256, smem);
}
template <int PER, bool VEC, int NB>
bool launch_backward_as(const BalArgs& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const size_t smem = RowRing<PER, VEC>::bytes();
  return prepare(k_bal_backward<PER, VEC, NB>, done, smem) &&
         launch(k_bal_backward<PER, VEC, NB>, row_blocks(a.T, backward_blocks<PER>()), stream, a, 256, smem);
}
template <int PER, bool VEC>
bool launch_backward(const BalArgs& a, cudaStream_t stream) {
  return a.k <= 8 ? launch_backward_as<PER, VEC, 4>(a, stream) : launch_backward_as<PER, VEC, 2>(a, stream);
}
bool one_block(const BalArgs& a) {
  return a.T <= ONE_TOKENS && a.n_seq <= ONE_TOKENS && (int64_t)a.T * a.E <= ONE_ELEMS && (int64_t)a.n_seq * a.E <= ONE_COUNTS;
}
template <int PER, bool VEC>
bool launch_one(const BalArgs& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  return prepare(k_bal_one<PER, VEC>, done, 0) && launch(k_bal_one<PER, VEC>, 1, stream, a, 1024);
}
// f(PER, VEC) for the row length: elements a lane holds, and whether rows are made of 16-byte pieces.
template <typename F>
bool by_row(int E, F f) {
  if (E % 4) return E <= 128 ? f(std::integral_constant<int, 4>(), std::false_type()) : f(std::integral_constant<int, 16>(), std::false_type());
  if (E <= 128) return f(std::integral_constant<int, 4>(), std::true_type());
  if (E <= 256) return f(std::integral_constant<int, 8>(), std::true_type());
  return f(std::integral_constant<int, 16>(), std::true_type());
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
  const size_t E4 = sizeof(float) * c->num_experts, n4 = sizeof(int) * (size_t)n_seq;
  if (overlap({{loss, 4}, {counts, E4}, {seq_counts, E4 * n_seq}, {seq_tokens, n4}, {ws, w.total}},
              {{logits, E4 * T}, {idx, sizeof(int) * (size_t)T * c->top_k}, {seq_start, n4 + 4}}))
    return FLINT_MOE_EINVAL;
  BalArgs a = {};
  a.T = T;
  a.E = c->num_experts;
  a.k = c->top_k;
  a.n_seq = n_seq;
  a.narrow = (int64_t)c->top_k * T * c->num_experts < ((int64_t)1 << 31);
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
  bool ok;
  if (one_block(a)) {
    ok = by_row(a.E, [&](auto per, auto vec) { return launch_one<per(), vec()>(a, stream); });
  } else {
    static std::atomic<uint64_t> zero_done{0}, count_done{0};
    ok = prepare(k_bal_zero, zero_done, 0) && prepare(k_bal_count, count_done, 0) &&
         launch(k_bal_zero, (int)std::min<size_t>(SMS, ((size_t)n_seq * a.E + 255) / 256), stream, a) &&
         (T == 0 || (launch(k_bal_count, std::min(COUNT_BLOCKS, (T + 255) / 256), stream, a) &&
                     by_row(a.E, [&](auto per, auto vec) { return launch_loss<per(), vec()>(a, stream); })));
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
  const size_t E4 = sizeof(float) * c->num_experts, k4 = sizeof(int) * (size_t)T * c->top_k, n4 = sizeof(int) * (size_t)n_seq;
  if (overlap({{dlogits, E4 * T}},
              {{logits, E4 * T}, {idx, k4}, {seq_start, n4 + 4}, {seq_counts, E4 * n_seq}, {seq_tokens, n4}, {dloss, 4}, {dw, k4}}))
    return FLINT_MOE_EINVAL;
  BalArgs a = {};
  a.T = T;
  a.E = c->num_experts;
  a.k = c->top_k;
  a.n_seq = n_seq;
  a.narrow = (int64_t)c->top_k * T * c->num_experts < ((int64_t)1 << 31);
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
  const bool ok = by_row(a.E, [&](auto per, auto vec) { return launch_backward<per(), vec()>(a, stream); });
  return ok ? FLINT_MOE_OK : FLINT_MOE_ECUDA;
}
