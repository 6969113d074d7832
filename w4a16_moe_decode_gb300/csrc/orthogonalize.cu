// Orthogonalised updates by Newton-Schulz steps (flint_orthogonalize.h), as matrix products of gemm.cuh, or in one kernel
// where a matrix fits a cluster's shared memory.
//
// A step's X <- a X + P X with P = b S + c S S, S = X X^T. What is added to X is amplified by the later steps where X is
// weak, by up to a^steps (485 after five steps of 3.4445): X is kept as hi + lo f16, or in FP32. An error
// relative to X from the left, (1 + e) X, only turns the result by e: so the products take f16 values, S from X's hi, P
// from one rounding of each of its parts, and the tensor cores run at one product's rate instead of three (few rows apart,
// below). S, P and the
// update of wide X read their transposes as they lie (S and P are their own); S and P are computed above the diagonal.
// Scaled values: X is kept times 2^10, S times 2^10 and P times 2^8, so that f16 holds X and S to 2^-35 and P to 2^-33, or to
// a relative 2^-11 (X's two values 2^-22) where that is more. A matrix whose norm is far below eps gives an X far below one:
// it is kept times a further power of two, which falls as the steps let X grow (Size).
//
// Two updates of 8192 x 2048, us: 980 (1130 TFLOP/s of the products that cannot be left out), bound by the tensor cores
// in X P and, in the two products of S, by one round of 72 tiles; norm and conversion take 60 of it from memory. 256 x
// 2048: 85, seventeen launches of 5 us that wait for one another.
#include <cmath>
#include <type_traits>

#include "flint_orthogonalize.h"
#include "gemm.cuh"

namespace flint {
namespace ortho {

using namespace gemm;

// X, S and P as two f16 values each up to 32 rows, and products of them as three (hi hi, hi lo, lo hi): few rounding errors
// meet in a result there, and a step multiplies a singular value's by up to 5 near 1.2 (with S as one value, 600 matrices of
// 2 rows were up to 0.0097 off and of 6 0.0045; so 0.0033 and 0.0024, what rounding them once gives. 8 of 16 x 2048: 23.8
// and 25.2 us). Up to 64 P alone is, where S is nearly diagonal for long matrices, so that one rounding of a place of P's
// diagonal turns a whole row (33 x 700 of noise: 0.0041 off with P_hi alone, 0.0025 so; 16 of 64 x 2048 40.7 and 41.7).
// Above, one value of each, whose errors average out (128 x 2000 of noise: 0.0024).
__host__ __device__ inline bool few_rows(int m) { return m <= 32; }
__host__ __device__ inline bool p_halves(int m) { return m <= 64; }

constexpr float X_SCALE = 1024.f, S_SCALE = 1024.f, P_SCALE = 256.f;

__device__ __forceinline__ uint32_t f2h2(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 h2f2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint4 pack8_f16(const float* v) {
  return make_uint4(f2h2(v[0], v[1]), f2h2(v[2], v[3]), f2h2(v[4], v[5]), f2h2(v[6], v[7]));
}
__device__ __forceinline__ void unpack8_f16(const uint4 u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = h2f2(w[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
// hi + lo = v to 22 bits.
__device__ __forceinline__ void split8(const float* v, uint4& hi, uint4& lo) {
  float h[8], l[8];
  hi = pack8_f16(v);
  unpack8_f16(hi, h);
#pragma unroll
  for (int i = 0; i < 8; ++i) l[i] = v[i] - h[i];
  lo = pack8_f16(l);
}

// ---------------------------------------------------------------------------
// X = M / (|M| + eps): the sums of squares (a thread's in FP32 with an exponent
// of its own, so that squares neither overflow nor vanish, the threads' and
// blocks' in FP64, of which this card computes two a cycle and SM), then hi and
// lo.
// ---------------------------------------------------------------------------
struct Start {
  const void* in;
  int bf16, n, rows, cols, pitch, parts;
  float eps;
  double* part;  // [n][parts]
  uint16_t *hi, *lo;
  int* status;
  int steps;
  float coeffs[3 * FLINT_ORTHOGONALIZE_MAX_STEPS];
  float4* factors;  // [n][FLINT_ORTHOGONALIZE_MAX_STEPS]: Size::Step of each step
};

// What X is kept times, 2^e, from a bound of its size, which a step raises to |a| n + |b| n^3 + |c| n^5 at most. So a small
// X fills f16's range as a large one does, its S and P with it, and the bound of a grown one ends at e = 0.
constexpr int SIZE_MOST = 100;  // (an X below 2^-100 keeps fewer digits)
__device__ __forceinline__ int exponent(float v) { return (int)(__float_as_uint(v) >> 23) - 127; }  // of v >= 0
struct Size {
  float n;  // bound of what is kept, 2^e X
  int e;
  // P = ps S + pq S S, X <- ua X + up P X, of what is kept of each.
  struct Step {
    float ps, pq, up, ua;
  };
  // The factors of a step; after the last one X is kept as it is.
  __device__ __forceinline__ Step next(float a, float b, float c, bool last) {
    const float w = exp2i(-e), t = n * w, t2 = t * t;
    const float n1 = fminf(n * (fabsf(a) + t2 * (fabsf(b) + fabsf(c) * t2)), 0x1p120f);
    const int e1 = last ? 0 : n1 > 0.f ? min(max(e - exponent(n1) - 1, 0), SIZE_MOST) : e;
    // P of a small X is 2^2e times its value: coefficients that f16 would not hold then are scaled down.
    const int pe = e > 0 ? max(exponent(fabsf(b) + fabsf(c) * w * w) - 6, 0) : 0;
    const Step s = {b * (P_SCALE / S_SCALE) * exp2i(-pe), c * (P_SCALE / (S_SCALE * S_SCALE)) * exp2i(max(-2 * e - pe, -126)),
                    (1.0f / P_SCALE) * exp2i(min(max(pe - 2 * e + e1 - e, -126), 126)), a * exp2i(e1 - e)};
    n = n1 * exp2i(e1 - e);
    e = e1;
    return s;
  }
};

constexpr int START_THREADS = 256;

__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(uint16_t v) { return bf16lo(v); }
// Eight values from an aligned place.
__device__ __forceinline__ void load8(const uint16_t* p, float* v) { unpack8_bf16(*reinterpret_cast<const uint4*>(p), v); }
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
  v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
}
__device__ __forceinline__ float load1(const Start& a, size_t i) {
  return a.bf16 ? value(static_cast<const uint16_t*>(a.in)[i]) : value(static_cast<const float*>(a.in)[i]);
}
// Values i .. i + 7 (i a multiple of 8 from an aligned start).
__device__ __forceinline__ void load8(const Start& a, size_t i, float* v) {
  if (a.bf16)
    load8(static_cast<const uint16_t*>(a.in) + i, v);
  else
    load8(static_cast<const float*>(a.in) + i, v);
}

// A sum of squares as q 4^ex: neither overflows nor vanishes.
struct Squares {
  float q = 0.f;
  int ex = -126;
  template <int N>
  __device__ __forceinline__ void add(const float (&v)[N]) {
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) mx = fmaxf(mx, fabsf(v[e]));
    const int to = min(max((int)(__float_as_uint(mx) >> 23) - 127, ex), 126);
    const float down = exp2i(max(ex - to, -126)), sc = exp2i(-to);
    q = q * down * down;
    ex = to;
#pragma unroll
    for (int e = 0; e < N; ++e) q = fmaf(v[e] * sc, v[e] * sc, q);
  }
  __device__ __forceinline__ double value() const { return (double)q * __longlong_as_double((long long)(1023 + 2 * ex) << 52); }
};
// 2^e X_SCALE / (|M| + eps) as two FP32 factors, since a large norm's is below FP32's normals, and X's size.
__device__ __forceinline__ float2 inverse(double sum, float eps, Size& size) {
  const double norm = sqrt(sum), d = norm + (double)eps;
  const int ed = (int)(__double_as_longlong(d) >> 52) - 1023, en = (int)(__double_as_longlong(norm) >> 52) - 1023, half = ed / 2;
  size = {1.0f, norm > 0.0 ? min(max(ed - en - 1, 0), SIZE_MOST) : 0};
  const int e0 = size.e / 2;
  return make_float2(exp2i(e0 - half), (float)(X_SCALE / (d * __longlong_as_double((long long)(1023 - half - (size.e - e0)) << 52))));
}

__global__ void __launch_bounds__(START_THREADS) k_ortho_norm(const Start a) {
  __shared__ double s_sum[START_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0 && blockIdx.x + blockIdx.y == 0) *a.status = 0;
  const size_t all = (size_t)a.rows * a.cols, first = blockIdx.y * all;
  const bool vec = all % 8 == 0;
  Squares sq;
  for (size_t i = 8 * ((size_t)blockIdx.x * START_THREADS + threadIdx.x); i < all; i += (size_t)gridDim.x * START_THREADS * 8) {
    float v[8];
    if (vec) {
      load8(a, first + i, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = i + e < all ? load1(a, first + i + e) : 0.f;
    }
    sq.add(v);
  }
  double sum = sq.value();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < START_THREADS / 32; ++w) sum += s_sum[w];
    a.part[(size_t)blockIdx.y * a.parts + blockIdx.x] = sum;
  }
}

__global__ void __launch_bounds__(START_THREADS) k_ortho_split(const Start a) {
  __shared__ float s_scale[2];
  Size size = {1.0f, 0};  // (thread 0)
  // The last block is for the steps' factors alone, which take as long as a block's share of a small matrix.
  const bool factors = blockIdx.x == a.parts;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 32) {
    double sum = 0.0;
    for (int p = threadIdx.x; p < a.parts; p += 32) sum += __ldcg(a.part + (size_t)blockIdx.y * a.parts + p);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (threadIdx.x == 0) {
      const float2 f = inverse(sum, a.eps, size);
      s_scale[0] = f.x;
      s_scale[1] = f.y;
    }
  }
  __syncthreads();
  const float s0 = s_scale[0], s1 = s_scale[1];
  if (factors) {
    if (threadIdx.x >= 32) return;
    auto step = [&](int i, Size& z) {
      const Size::Step s = z.next(a.coeffs[3 * i], a.coeffs[3 * i + 1], a.coeffs[3 * i + 2], i + 1 == a.steps);
      a.factors[(size_t)blockIdx.y * FLINT_ORTHOGONALIZE_MAX_STEPS + i] = make_float4(s.ps, s.pq, s.up, s.ua);
    };
    const int i = threadIdx.x;
    const bool mine = i < a.steps, grows = !mine || fabsf(a.coeffs[3 * i]) >= 1.0f;
    if (__all_sync(0xffffffffu, grows) && __shfl_sync(0xffffffffu, size.e, 0) == 0) {  // kept as it is in every step
      size = {1.0f, 0};
      if (mine) step(i, size);
    } else if (i == 0) {
      for (int k = 0; k < a.steps; ++k) step(k, size);
    }
    return;
  }
  const size_t all = (size_t)a.rows * a.cols, first = blockIdx.y * all, out = (size_t)blockIdx.y * a.rows * a.pitch;
  const size_t step = (size_t)a.parts * START_THREADS;
  if (a.pitch == a.cols) {  // rows of whole pieces of eight
    for (size_t i = 8 * ((size_t)blockIdx.x * START_THREADS + threadIdx.x); i < all; i += 8 * step) {
      float v[8];
      load8(a, first + i, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (v[e] * s0) * s1;
      uint4 hi, lo;
      split8(v, hi, lo);
      *reinterpret_cast<uint4*>(a.hi + out + i) = hi;
      *reinterpret_cast<uint4*>(a.lo + out + i) = lo;
    }
  } else {
    // a warp a row, each lane up to eight of its values at a time
    const int lane = threadIdx.x & 31, warps = a.parts * (START_THREADS / 32);
    for (int r = blockIdx.x * (START_THREADS / 32) + (threadIdx.x >> 5); r < a.rows; r += warps) {
      const size_t from = first + (size_t)r * a.cols, to = out + (size_t)r * a.pitch;
      for (int c0 = lane; c0 < a.cols; c0 += 256) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c0 + 32 * e < a.cols ? load1(a, from + c0 + 32 * e) : 0.f;
        uint4 hi, lo;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (v[e] * s0) * s1;
        split8(v, hi, lo);
        const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c0 + 32 * e < a.cols) {
            a.hi[to + c0 + 32 * e] = (uint16_t)(e & 1 ? h[e >> 1] >> 16 : h[e >> 1]);
            a.lo[to + c0 + 32 * e] = (uint16_t)(e & 1 ? l[e >> 1] >> 16 : l[e >> 1]);
          }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Epilogues: S, P = b S + c S S, X <- a X + P X.
// ---------------------------------------------------------------------------
template <bool LO>  // S's second half too (few_rows: one tile a matrix)
struct Gram {
  static constexpr bool PAIR = false, SMALL = LO;
  static constexpr int MAPS = 1, OUTS = LO ? 2 : 1, INS = 0;
  struct Args {};
  using Pre = NoPre;
  static __device__ __forceinline__ void matrix(const Args&, Part&) {}
  static __device__ __forceinline__ void chunk(const Args&, const MapsOf<Gram>& maps, Part& t, int c, uint32_t (&w)[32], uint32_t (&)[32],
                                               const Pre&) {
    float* v = reinterpret_cast<float*>(w);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= S_SCALE / (X_SCALE * X_SCALE);
    const uint4 o[4] = {pack8_f16(v), pack8_f16(v + 8), pack8_f16(v + 16), pack8_f16(v + 24)};
    t.put(&maps.io[0], t.n0 + c, o);
    if (t.twice) t.put_transposed(&maps.io[0], t.n0 + c, o);
    if constexpr (LO) {
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float2 hi = h2f2(f2h2(v[j], v[j + 1]));
        v[j] -= hi.x, v[j + 1] -= hi.y;
      }
      const uint4 l[4] = {pack8_f16(v), pack8_f16(v + 8), pack8_f16(v + 16), pack8_f16(v + 24)};
      t.put(&maps.io[1], t.n0 + c, l);
    }
  }
};

// 32 columns of this lane's row of a matrix [batch][M][pitch], from the tile's column c on; zero outside.
__device__ __forceinline__ void load_row(const Part& t, const uint16_t* m, int pitch, int c, uint4 (&v)[4]) {
  const uint16_t* at = m + ((size_t)t.z * t.M + t.row) * pitch + t.n0 + c;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = t.row < t.M && t.n0 + c + 8 * j < t.N ? __ldcg(reinterpret_cast<const uint4*>(at + 8 * j)) : make_uint4(0, 0, 0, 0);
}

// A matrix's factors of a step, which k_ortho_split left.
__device__ __forceinline__ float4 factors_of(const float4* f, int z) { return __ldcg(f + (size_t)z * FLINT_ORTHOGONALIZE_MAX_STEPS); }

template <bool LO>  // S's second half (few_rows)
struct Poly {
  static constexpr bool PAIR = false, SMALL = LO;
  static constexpr int MAPS = 1, OUTS = 2, INS = LO ? 2 : 1;
  struct Args {
    const uint16_t *s, *s_lo;
    int pitch;
    const float4* factors;  // of this step, FLINT_ORTHOGONALIZE_MAX_STEPS apart
    int lo;                 // P's second half too (p_halves)
  };
  struct Pre {
    uint4 s[4], l[LO ? 4 : 1];
    __device__ __forceinline__ Pre(const Args& a, const Part& t, int c) {
      load_row(t, a.s, a.pitch, c, s);
      if constexpr (LO) load_row(t, a.s_lo, a.pitch, c, l);
    }
    __device__ __forceinline__ Pre(const Part& t, const uint8_t* in) {
      slot_row(t, in, s);
      if constexpr (LO) slot_row(t, in + SLOT, l);
    }
  };
  static __device__ __forceinline__ void matrix(const Args& a, Part& t) { t.f = factors_of(a.factors, t.z); }
  static __device__ __forceinline__ void chunk(const Args& a, const MapsOf<Poly>& maps, Part& t, int c, uint32_t (&w)[32], uint32_t (&)[32],
                                               const Pre& pre) {
    const float fs = t.f.x, fq = t.f.y;
    uint4 hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[8];
      unpack8_f16(pre.s[j], v);
      if constexpr (LO) {
        float l[8];
        unpack8_f16(pre.l[j], l);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += l[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(fs, v[i], fq * __uint_as_float(w[8 * j + i]));
      split8(v, hi[j], lo[j]);
    }
    t.put(&maps.io[0], t.n0 + c, hi);
    if (t.twice) t.put_transposed(&maps.io[0], t.n0 + c, hi);
    if (a.lo) {
      t.put(&maps.io[1], t.n0 + c, lo);
      if (t.twice) t.put_transposed(&maps.io[1], t.n0 + c, lo);
    }
  }
};

template <bool LAST>
struct Update {
  static constexpr bool PAIR = false, SMALL = false;
  static constexpr int MAPS = 1, OUTS = 2, INS = 2;
  struct Args {
    const uint16_t *hi, *lo;
    int pitch;
    const float4* factors;
    float scale;
    uint16_t* out;  // LAST: [batch][M][N]
  };
  struct Pre {
    uint4 hi[4], lo[4];
    __device__ __forceinline__ Pre(const Args& a, const Part& t, int c) {
      load_row(t, a.hi, a.pitch, c, hi);
      load_row(t, a.lo, a.pitch, c, lo);
    }
    __device__ __forceinline__ Pre(const Part& t, const uint8_t* in) {
      slot_row(t, in, hi);
      slot_row(t, in + SLOT, lo);
    }
  };
  static __device__ __forceinline__ void matrix(const Args& a, Part& t) { t.f = factors_of(a.factors, t.z); }
  static __device__ __forceinline__ void chunk(const Args& a, const MapsOf<Update>& maps, Part& t, int c, uint32_t (&w)[32], uint32_t (&)[32],
                                               const Pre& pre) {
    const float fp = t.f.z, fa = t.f.w;
    uint4 hv[4], lv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float h[8], l[8], v[8];
      unpack8_f16(pre.hi[j], h);
      unpack8_f16(pre.lo[j], l);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(fp, __uint_as_float(w[8 * j + i]), fa * (h[i] + l[i]));
      if (LAST) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= a.scale;
        hv[j] = pack8_bf16(v);
      } else {
        split8(v, hv[j], lv[j]);
      }
    }
    if (!LAST || t.N % 8 == 0) {
      t.put(&maps.io[0], t.n0 + c, hv);
      if (!LAST) t.put(&maps.io[1], t.n0 + c, lv);
    } else {  // rows that TMA cannot reach: through a slot, a row's neighbours by neighbouring lanes
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(t.sm + Part::piece(t.lane, j)) = hv[j];
      __syncwarp();
      const int col = t.n0 + c + t.lane;
      for (int r = 0; r < 32 && t.row0 + r < t.M; ++r)
        if (col < t.N)
          a.out[((size_t)t.z * t.M + t.row0 + r) * t.N + col] =
              *reinterpret_cast<const uint16_t*>(t.sm + Part::piece(r, t.lane >> 3) + (t.lane & 7) * 2);
    }
  }
};

// ---------------------------------------------------------------------------
// Few rows (the shorter side up to 128) that fit the shared memory of a cluster:
// all steps in one kernel, one cluster of CTAs a matrix. The matrix lies on its
// long side here, X [k][m] with m <= 128: each CTA keeps kc of the k rows, in
// FP32 in its threads' registers and as f16 in the swizzled layout in which the
// same bytes serve as both operands of S = X^T X (MN-major, the rows being the
// reduction) and as X in X P (K-major). A step:
//   S's partial sums of the CTA's rows (tcgen05) -> shared memory; each CTA adds
//   its share of them over the cluster and hands the f16 result to all;
//   P = b S + c S S, by every CTA for itself;
//   X <- a X + X P, by rows (few_rows, p_halves: with the second halves of X, S and P).
// Bound by latency: two cluster barriers, the exchange between them and three
// products that wait for one another a step. 8 matrices of 16 x 2048: 105 us
// with the general path's 17 launches, 25 here; 16 of 64 x 2048 183 and 42;
// four of 128 x 2048 140 and 52. Tried: clusters of eight for 64 rows (one matrix
// 47 us, 16 in two rounds 94), X in shared memory as hi and lo alone (63), the
// sums read in rank order (the exchange 14500 cycles instead of 6300).
// ---------------------------------------------------------------------------
constexpr int FEW_THREADS = 512;
constexpr int FEW_GROUPS = FEW_THREADS / 128;  // four warps reach all of tensor memory's lanes
constexpr uint32_t S_LO = 64 * 128;            // S's second half (few_rows): the rows of its box from 64 on
constexpr int FEW_UNITS = 4;                   // of 16 columns of a row, that a thread keeps at most (128 registers, up to 32 words spilt)

struct FewArgs {
  const void* in;
  uint16_t* out;
  int bf16, rows, cols, steps;
  int m, k, kc;  // the shorter and the longer side, rows of the long side a CTA keeps (multiple of 128)
  float eps, scale;
  float coeffs[3 * FLINT_ORTHOGONALIZE_MAX_STEPS];
  int* status;
};

struct FewPlan {
  int mp, mb, xbox, sbox, pbox, sums, tmem;  // columns padded to 16, boxes of 64; bytes of a box of X, S, P and of sums; tensor memory
  size_t x[2], s, p, total;            // x: hi, lo; p: P's halves, and S's partial sums before
};
__host__ __device__ inline FewPlan few_plan(int m, int kc) {
  FewPlan f;
  f.mp = (m + 15) & ~15;
  f.mb = m > 64 ? 2 : 1;
  f.xbox = kc * 128;
  f.sbox = 128 * 128;
  f.pbox = f.mb == 1 ? 64 * 128 : 128 * 128;
  const int halves = few_rows(m) ? 2 : 1;
  f.x[0] = 0;
  f.x[1] = (size_t)(halves - 1) * f.mb * f.xbox;
  f.s = (size_t)halves * f.mb * f.xbox;
  f.p = f.s + (size_t)f.mb * f.sbox;
  f.sums = f.mp * m * 4;
  const size_t p = (size_t)(p_halves(m) ? 2 : 1) * f.mb * f.pbox, sums = (size_t)halves * f.sums;
  f.total = 1024 + f.p + (p > sums ? p : sums);
  const int cols = (kc / 128 + 2) * f.mp;
  f.tmem = cols <= 64 ? 64 : cols <= 128 ? 128 : cols <= 256 ? 256 : 512;
  return f;
}
// Units a thread keeps.
__host__ __device__ inline int few_units(int m, int kc) { return (kc / 128 * ((m + 15) / 16) + FEW_GROUPS - 1) / FEW_GROUPS; }

__device__ __forceinline__ void st_dsmem_v4(uint32_t remote, const uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(remote), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ double ld_dsmem_f64(uint32_t remote) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(remote) : "memory");
  return v;
}
// What 16 ks columns of a K-major operand in boxes of 64 columns add to its descriptor.
__device__ __forceinline__ uint32_t k_step(int ks, int box) { return (uint32_t)((ks >> 2) * (box >> 4) + (ks & 3) * 2); }

template <int UNITS, bool BOTH>  // (few_rows)
__global__ void __launch_bounds__(FEW_THREADS, 1) k_ortho_few(const FewArgs a) {
  extern __shared__ uint8_t dsmem[];
  __shared__ double s_sum[FEW_THREADS / 32], s_part;
  __shared__ float2 s_inv;
  __shared__ Size::Step s_step;
  __shared__ uint64_t bar;
  __shared__ uint32_t tmem_base;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, group = warp >> 2;
  const int C = gridDim.x, rank = blockIdx.x;
  const FewPlan f = few_plan(a.m, a.kc);
  const bool both_p = BOTH || p_halves(a.m);
  const uint32_t base = (smem_addr(dsmem) + 1023u) & ~1023u;
  uint8_t* const sm = dsmem + (base - smem_addr(dsmem));
  const uint32_t xs = base + (uint32_t)f.x[0], xls = base + (uint32_t)f.x[1], ss = base + (uint32_t)f.s, ps = base + (uint32_t)f.p;
  uint8_t *const xp = sm + f.x[0], *const xlp = sm + f.x[1], *const sp = sm + f.s, *const pp = sm + f.p;
  const int plo = f.mb * f.pbox;  // P's second half behind the first
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&tmem_base, f.tmem);
  for (int i = threadIdx.x; i < f.mb * f.sbox / 16; i += FEW_THREADS) reinterpret_cast<uint4*>(sp)[i] = make_uint4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  Size size;  // (this thread's: not one of the warp that issues the products)
  const bool sizes = threadIdx.x == FEW_THREADS - 32;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0 && blockIdx.x + blockIdx.y == 0) *a.status = 0;

  // Unit n of this thread: row 128 t + i0 of the CTA's, columns c .. c + 15. The matrix as it lies in memory has X's rows
  // down (tall) or across.
  const bool tall = a.rows > a.cols, vec = tall && a.cols % 8 == 0;
  const int chunks = f.mp / 16, tiles = a.kc / 128, i0 = q * 32 + lane, l0 = rank * a.kc;
  const size_t first = (size_t)blockIdx.y * a.rows * a.cols;
  auto unit = [&](int n, int& t, int& c) {
    const int u = group + n * FEW_GROUPS;
    t = u / chunks;
    c = (u - t * chunks) * 16;
    return u < tiles * chunks;
  };
  auto xoff = [&](int l, int pc) { return (uint32_t)((pc >> 3) * f.xbox + l * 128 + (((pc & 7) ^ (l & 7)) << 4)); };
  float x[UNITS][16];
  auto load = [&](auto* in) {  // float or bf16 bits
    using T = std::remove_const_t<std::remove_pointer_t<decltype(in)>>;
#pragma unroll
    for (int n = 0; n < UNITS; ++n) {
      int t, c;
      const bool live = unit(n, t, c);
      const int at = l0 + t * 128 + i0, most = live && at < a.k ? a.m - c : 0;  // columns that there are
      const size_t step = tall ? 1 : a.cols;
      const T* p = in + first + (tall ? (size_t)at * a.cols : (size_t)at) + (size_t)c * step;
      if (vec) {
#pragma unroll
        for (int h = 0; h < 16; h += 8) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[n][h + e] = 0.f;
          if (h < most) load8(p + h, &x[n][h]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[n][e] = e < most ? value(p[e * step]) : 0.f;
      }
    }
  };
  if (a.bf16)
    load(static_cast<const uint16_t*>(a.in));
  else
    load(static_cast<const float*>(a.in));
  Squares sq;
#pragma unroll
  for (int n = 0; n < UNITS; ++n) sq.add(x[n]);
  double sum = sq.value();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < FEW_THREADS / 32; ++w) sum += s_sum[w];
    s_part = sum;
  }
  cluster_sync();
  if (sizes) {
    sum = 0.0;
    for (int r = 0; r < C; ++r) sum += ld_dsmem_f64(dsmem_addr(smem_addr(&s_part), r));
    s_inv = inverse(sum, a.eps, size);
  }
  __syncthreads();
  const float2 inv = s_inv;
  // Unit n's f16 values to where the products read them.
  auto hand_over = [&](int n, int t, int c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t o = xoff(t * 128 + i0, c / 8 + h);
      if constexpr (BOTH) {
        uint4 hi, lo;
        split8(&x[n][8 * h], hi, lo);
        *reinterpret_cast<uint4*>(xp + o) = hi;
        *reinterpret_cast<uint4*>(xlp + o) = lo;
      } else {
        *reinterpret_cast<uint4*>(xp + o) = pack8_f16(&x[n][8 * h]);
      }
    }
  };
#pragma unroll
  for (int n = 0; n < UNITS; ++n) {
    int t, c;
    if (!unit(n, t, c)) break;
#pragma unroll
    for (int e = 0; e < 16; ++e) x[n][e] = (x[n][e] * inv.x) * inv.y;
    hand_over(n, t, c);
  }

  const uint32_t d_s = tmem, d_q = tmem + f.mp, d_x = tmem + 2 * f.mp;  // S, S S, and X P by tiles of 128 rows
  const uint32_t lanes = (uint32_t)(q * 32) << 16;
  const int swz = f.mp % 32 == 0 ? 7 : 3;
  uint32_t phase = 0;
  bool ok = true;
  auto arrived = [&] {  // the products asked for last; after a wait that gave up the others are not waited for
    ok = ok && mbar_wait(&bar, phase, a.status);
    phase ^= 1;
    __syncwarp();
    tc_fence_after();
  };
  auto ready = [&] {  // all threads have written their shared memory and read their tensor memory
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };
  // The thread that issues a product orders what it has seen the others write before the tensor core's reads of it.
  for (int step = 0; step < a.steps; ++step) {
    ready();
    if (sizes) s_step = size.next(a.coeffs[3 * step], a.coeffs[3 * step + 1], a.coeffs[3 * step + 2], step + 1 == a.steps);
    if (warp == 0 && elect_one()) {
      fence_proxy_async();
      // With one box of columns, rows of D from 64 on come from X's lo (BOTH), or, not read, from eight rows of X further
      // on, and at the end from the 1 KiB behind X, which is S's: a second box's place could lie outside the shared memory.
      const uint32_t idesc = idesc_f32acc(128, f.mp, false) | IDESC_A_MN | IDESC_B_MN;
      uint64_t d = sw128_desc_mn(xs, f.mb == 1 && !BOTH ? 1024 : f.xbox);
#pragma unroll 4
      for (int ks = 0; ks < a.kc / 16; ++ks, d += 2048 >> 4) tc_mma(d_s, d, d, idesc, ks > 0);
      tc_commit(&bar);
    }
    __syncwarp();
    arrived();
    // This CTA's sums, by rows, pieces of four swizzled by row; those of X's lo behind them.
    const bool lo_row = BOTH && i0 >= 64;
    const int si = lo_row ? i0 - 64 : i0;
    uint8_t* const sums = pp + (lo_row ? f.sums : 0);
    for (int c = 16 * group; c < f.mp; c += 16 * FEW_GROUPS) {
      uint32_t w[16];
      __syncwarp();
      tc_ld16(d_s + lanes + c, w);
      if (si < a.m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(sums + (si * (f.mp / 4) + ((c / 4 + j) ^ (si & swz))) * 16) =
              make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    }
    tc_fence_before();
    if constexpr (BOTH) {  // S = hi hi + lo hi + hi lo, the last the transpose of the one before
      __syncthreads();
      auto place = [&](int i, int n) { return (uint32_t)((i * (f.mp / 4) + ((n >> 2) ^ (i & swz))) * 16 + (n & 3) * 4); };
      const uint8_t* const lo = pp + f.sums;
      for (int i = threadIdx.x >> (f.mp == 16 ? 4 : 5), n = threadIdx.x & (f.mp - 1); i < a.m; i += FEW_THREADS / f.mp) {
        if (n < a.m)
          *reinterpret_cast<float*>(pp + place(i, n)) +=
              *reinterpret_cast<const float*>(lo + place(i, n)) + *reinterpret_cast<const float*>(lo + place(n, i));
      }
    }
    __syncwarp();
    cluster_sync();
    {
      // Pieces of four columns, neighbouring threads a row's; two threads join theirs to one piece of eight f16 values and
      // hand it to half of the CTAs each. A CTA begins with its own sums and goes round, so that no CTA's memory is asked
      // by all at once.
      const int per = f.mp / 4, all = f.mp / 8 * a.m, e1 = 2 * (all * (rank + 1) / C);
      for (int e0 = 2 * (all * rank / C) + warp * 32; e0 < e1; e0 += FEW_THREADS) {
        const int e = min(e0 + lane, e1 - 1), i = e / per, c = e - i * per;
        const uint32_t at = ps + (uint32_t)(i * per + (c ^ (i & swz))) * 16;
        float4 p[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < C) p[r] = ld_dsmem_f4(dsmem_addr(at, (rank + r) & (C - 1)));
        float4 v = p[0];
#pragma unroll
        for (int r = 1; r < 8; ++r)
          if (r < C) v.x += p[r].x, v.y += p[r].y, v.z += p[r].z, v.w += p[r].w;
        constexpr float fs = S_SCALE / (X_SCALE * X_SCALE);
        v.x *= fs, v.y *= fs, v.z *= fs, v.w *= fs;
        // (returns what the f16 values leave)
        auto give = [&](const float4 u, uint32_t to) {
          const uint32_t w0 = f2h2(u.x, u.y), w1 = f2h2(u.z, u.w);
          const uint32_t o0 = __shfl_xor_sync(0xffffffffu, w0, 1), o1 = __shfl_xor_sync(0xffffffffu, w1, 1);
          const uint4 o = lane & 1 ? make_uint4(o0, o1, w0, w1) : make_uint4(w0, w1, o0, o1);
          if (e0 + lane < e1)
            for (int r = lane & 1; r < C; r += 2) st_dsmem_v4(dsmem_addr(to, (rank + r) & (C - 1)), o);
          const float2 x = h2f2(w0), y = h2f2(w1);
          return make_float4(u.x - x.x, u.y - x.y, u.z - y.x, u.w - y.y);
        };
        const uint32_t to = ss + (uint32_t)((c >> 4) * f.sbox + i * 128 + ((((c >> 1) & 7) ^ (i & 7)) << 4));
        const float4 rest = give(v, to);
        if constexpr (BOTH) give(rest, to + S_LO);
      }
    }
    cluster_sync();
    tc_fence_after();
    if (warp == 0 && elect_one()) {
      fence_proxy_async();
      const uint32_t idesc = idesc_f32acc(128, f.mp, false);
      // (S's lo as A takes its rows from 64 on, which are not read, from behind S: P's place, which is as long)
      const uint64_t d = sw128_desc(ss), dl = sw128_desc(ss + S_LO);
#pragma unroll 4
      for (int ks = 0; ks < f.mp / 16; ++ks) {
        const uint32_t o = k_step(ks, f.sbox);
        tc_mma(d_q, d + o, d + o, idesc, ks > 0);
        if constexpr (BOTH) {
          tc_mma(d_q, dl + o, d + o, idesc, 1);
          tc_mma(d_q, d + o, dl + o, idesc, 1);
        }
      }
      tc_commit(&bar);
    }
    __syncwarp();
    arrived();
    const float fs = s_step.ps, fq = s_step.pq;
    for (int c = 16 * group; c < f.mp; c += 16 * FEW_GROUPS) {
      uint32_t w[16];
      __syncwarp();
      tc_ld16(d_q + lanes + c, w);
      if (i0 < f.mp)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int pc = c / 8 + j;
          float v[8];
          const uint32_t at = (uint32_t)(i0 * 128 + (((pc & 7) ^ (i0 & 7)) << 4));
          unpack8_f16(*reinterpret_cast<const uint4*>(sp + (pc >> 3) * f.sbox + at), v);
          if constexpr (BOTH) {
            float lo[8];
            unpack8_f16(*reinterpret_cast<const uint4*>(sp + S_LO + at), lo);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += lo[e];
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = fmaf(fs, v[e], fq * __uint_as_float(w[8 * j + e]));
          uint4 hi, lo;
          split8(v, hi, lo);
          *reinterpret_cast<uint4*>(pp + (pc >> 3) * f.pbox + at) = hi;
          if (both_p) *reinterpret_cast<uint4*>(pp + plo + (pc >> 3) * f.pbox + at) = lo;
        }
    }
    ready();
    if (warp == 0 && elect_one()) {
      fence_proxy_async();
      const uint32_t idesc = idesc_f32acc(128, f.mp, false);
      const uint64_t dh = sw128_desc(xs), dl = sw128_desc(xls), ph = sw128_desc(ps), pl = sw128_desc(ps + plo);
      for (int t = 0; t < tiles; ++t) {
        const uint32_t row = (uint32_t)t * (128 * 128 >> 4);
#pragma unroll 4
        for (int ks = 0; ks < f.mp / 16; ++ks) {
          const uint32_t ox = row + k_step(ks, f.xbox), op = k_step(ks, f.pbox);
          tc_mma(d_x + t * f.mp, dh + ox, ph + op, idesc, ks > 0);
          if (both_p) tc_mma(d_x + t * f.mp, dh + ox, pl + op, idesc, 1);
          if constexpr (BOTH) tc_mma(d_x + t * f.mp, dl + ox, ph + op, idesc, 1);
        }
      }
      tc_commit(&bar);
    }
    __syncwarp();
    const float fp = s_step.up, fa = s_step.ua;
    arrived();
#pragma unroll
    for (int n = 0; n < UNITS; ++n) {
      int t, c;
      if (!unit(n, t, c)) break;
      uint32_t w[16];
      tc_ld16(d_x + lanes + t * f.mp + c, w);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[n][e] = fmaf(fp, __uint_as_float(w[e]), fa * x[n][e]);
      if (step + 1 < a.steps) hand_over(n, t, c);
    }
  }
#pragma unroll
  for (int n = 0; n < UNITS; ++n) {
    int t, c;
    if (!unit(n, t, c)) break;
    const int at = l0 + t * 128 + i0;
    if (at >= a.k) continue;
#pragma unroll
    for (int e = 0; e < 16; ++e) x[n][e] *= a.scale;
#pragma unroll
    for (int h = 0; h < 16; h += 8) {
      const uint4 o = pack8_bf16(&x[n][h]);
      if (vec) {
        if (c + h < a.m) *reinterpret_cast<uint4*>(a.out + first + (size_t)at * a.cols + c + h) = o;
        continue;
      }
      const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
      const size_t step = tall ? 1 : a.cols, from = first + (tall ? (size_t)at * a.cols : (size_t)at) + (size_t)(c + h) * step;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + h + e < a.m) a.out[from + e * step] = (uint16_t)(e & 1 ? ow[e >> 1] >> 16 : ow[e >> 1]);
    }
  }
  if (!ok) mbar_drain(&bar, phase ^ 1);  // products may still be under way
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing of the other CTAs' still reads or writes this one's memory
  if (warp == 0) {
    tc_fence_after();
    tmem_free(tmem, f.tmem);
  }
}

}  // namespace ortho
}  // namespace flint

using namespace flint;
using namespace flint::ortho;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
constexpr int H_STATUS = 1;  // word of the header that flint_moe_read_status reads

bool supported(int n, int rows, int cols) {
  return n >= 0 && n <= FLINT_ORTHOGONALIZE_MAX_MATRICES && rows >= 1 && cols >= 1 &&
         std::max(rows, cols) <= FLINT_ORTHOGONALIZE_MAX_SIDE && std::min(rows, cols) <= 16384;
}

// Blocks of a matrix in the first two kernels: four pieces of eight values a thread, 1024 at most.
int parts_of(int rows, int cols) {
  const int64_t per = 4 * 8 * START_THREADS;
  return (int)std::min<int64_t>(1024, ((int64_t)rows * cols + per - 1) / per);
}

struct WsPlan {
  int m, pitch, mpitch, parts;
  size_t part, factors, x[2][2], s[2], p[2], total;  // x: of even and odd steps; x, s, p: hi and lo
};
WsPlan ws_plan(int n, int rows, int cols) {
  WsPlan w = {};
  w.m = std::min(rows, cols);
  w.pitch = (cols + 7) & ~7;
  w.mpitch = (w.m + 7) & ~7;
  w.parts = parts_of(rows, cols);
  const size_t xb = ws_align((size_t)2 * n * rows * w.pitch), mb = ws_align((size_t)2 * n * w.m * w.mpitch);
  size_t o = 256;
  w.part = o;
  o += ws_align(sizeof(double) * n * w.parts);
  w.factors = o;
  o += ws_align(sizeof(float4) * FLINT_ORTHOGONALIZE_MAX_STEPS * n);
  for (int i = 0; i < 4; ++i) {
    w.x[i >> 1][i & 1] = o;
    o += xb;
  }
  for (int i = 0; i < 2; ++i) {
    w.s[i] = o;
    o += i == 0 || few_rows(w.m) ? mb : 0;
  }
  for (int i = 0; i < 2; ++i) {
    w.p[i] = o;
    o += i == 0 || p_halves(w.m) ? mb : 0;
  }
  w.total = o;
  return w;
}

// The cluster kernel's CTAs a matrix and their rows of the long side, or 0 where a matrix does not fit eight of them. By
// the shape alone, so that a matrix has the same bits in every batch.
int few_ctas(int m, int k, int* kc) {
  if (m > 128) return 0;
  for (int C = 1; C <= 8; C *= 2) {
    *kc = ((k + C - 1) / C + 127) / 128 * 128;
    if (few_units(m, *kc) <= FEW_UNITS && *kc <= 1024 && few_plan(m, *kc).total <= 226 * 1024 && (*kc / 128 + 2) * few_plan(m, *kc).mp <= 512) return C;
  }
  return 0;
}

template <int UNITS, bool BOTH>
bool run_few(const FewArgs& a, int C, int n, cudaStream_t stream) {
  return launch<k_ortho_few<UNITS, BOTH>, 226 * 1024>(dim3(C, n), FEW_THREADS, few_plan(a.m, a.kc).total, C, stream, a);
}

bool overlaps(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np;
}

}  // namespace

extern "C" size_t flint_orthogonalize_workspace_bytes(int32_t n, int32_t rows, int32_t cols) {
  return n > 0 && supported(n, rows, cols) ? ws_plan(n, rows, cols).total : 0;
}

extern "C" flint_moe_status flint_orthogonalize(const void* in, int32_t fmt, int32_t n, int32_t rows, int32_t cols,
                                                const float* coeffs, int32_t steps, float eps, float scale, uint16_t* out,
                                                void* ws, size_t ws_size, cudaStream_t stream) {
  if (!supported(n, rows, cols) || (fmt != FLINT_ORTHOGONALIZE_F32 && fmt != FLINT_ORTHOGONALIZE_BF16))
    return FLINT_MOE_EUNSUPPORTED;
  if (!coeffs || steps < 1 || steps > FLINT_ORTHOGONALIZE_MAX_STEPS || !(eps > 0.f) || !std::isfinite(eps) || !std::isfinite(scale))
    return FLINT_MOE_EINVAL;
  for (int i = 0; i < 3 * steps; ++i)
    if (!std::isfinite(coeffs[i])) return FLINT_MOE_EINVAL;
  if (n == 0) return FLINT_MOE_OK;
  if (!in || !out || !ws) return FLINT_MOE_EINVAL;
  if (!aligned(in, 16) || !aligned(out, 16) || !aligned(ws, 256)) return FLINT_MOE_EALIGN;
  const WsPlan w = ws_plan(n, rows, cols);
  const size_t values = (size_t)n * rows * cols;
  if (ws_size < w.total || overlaps(ws, w.total, in, values * (fmt == FLINT_ORTHOGONALIZE_F32 ? 4 : 2)) ||
      overlaps(ws, w.total, out, values * 2))
    return FLINT_MOE_EINVAL;
  // out may be in, value for value; another overlap would let a matrix's result fall on one that is still to be read
  if (overlaps(in, values * (fmt == FLINT_ORTHOGONALIZE_F32 ? 4 : 2), out, values * 2) &&
      (fmt == FLINT_ORTHOGONALIZE_F32 || in != out))
    return FLINT_MOE_EINVAL;
  uint8_t* wsp = static_cast<uint8_t*>(ws);
  int* status = reinterpret_cast<int*>(ws) + H_STATUS;
  int kc = 0;
  bool ok = true;
  if (const int C = few_ctas(w.m, std::max(rows, cols), &kc)) {
    FewArgs a = {in, out, fmt == FLINT_ORTHOGONALIZE_BF16, rows, cols, steps, w.m, std::max(rows, cols), kc, eps, scale / X_SCALE, {}, status};
    std::copy(coeffs, coeffs + 3 * steps, a.coeffs);
    const int units = few_units(w.m, kc);
    if (few_rows(w.m))
      ok = units <= 1 ? run_few<1, true>(a, C, n, stream) : units <= 2 ? run_few<2, true>(a, C, n, stream) : run_few<4, true>(a, C, n, stream);
    else
      ok = units <= 1 ? run_few<1, false>(a, C, n, stream) : units <= 2 ? run_few<2, false>(a, C, n, stream) : run_few<4, false>(a, C, n, stream);
    return ok ? FLINT_MOE_OK : FLINT_MOE_ECUDA;
  }
  auto at = [&](size_t o) { return reinterpret_cast<uint16_t*>(wsp + o); };
  const bool tall = rows > cols;
  const int m = w.m;
  CUtensorMap x[2][2], xout[2][2], s[2], sout[2], p[2], pout[2], o;
  auto map = [&](CUtensorMap* mp, size_t off, int64_t c, int64_t r, int64_t pitch, bool as_out) {
    return map_matrix(mp, at(off), c, r, pitch, n, r * pitch, as_out);
  };
  for (int i = 0; i < 2; ++i) {
    ok = ok && map(&s[i], w.s[i], m, m, w.mpitch, false) && map(&sout[i], w.s[i], m, m, w.mpitch, true);
    for (int h = 0; h < 2; ++h)
      ok = ok && map(&x[i][h], w.x[i][h], cols, rows, w.pitch, false) && map(&xout[i][h], w.x[i][h], cols, rows, w.pitch, true);
    ok = ok && map(&p[i], w.p[i], m, m, w.mpitch, false) && map(&pout[i], w.p[i], m, m, w.mpitch, true);
  }
  o = sout[0];
  if (cols % 8 == 0) ok = ok && map_matrix(&o, out, cols, rows, cols, n, (int64_t)rows * cols, true);
  if (!ok) return FLINT_MOE_ECUDA;
  Start st = {in, fmt == FLINT_ORTHOGONALIZE_BF16, n, rows, cols, w.pitch, w.parts, eps,
                    reinterpret_cast<double*>(wsp + w.part), at(w.x[0][0]), at(w.x[0][1]), status, steps, {}, reinterpret_cast<float4*>(wsp + w.factors)};
  std::copy(coeffs, coeffs + 3 * steps, st.coeffs);
  const unsigned parts = (unsigned)w.parts, mats = (unsigned)n;
  if (!launch<k_ortho_norm, 0>(dim3(parts, mats), START_THREADS, 0, 0, stream, st) ||
      !launch<k_ortho_split, 0>(dim3(parts + 1, mats), START_THREADS, 0, 0, stream, st))
    return FLINT_MOE_ECUDA;
  const int kx = ((tall ? rows : cols) + BK - 1) / BK, km = (m + BK - 1) / BK;
  AllMaps<Gram<false>> mg;
  AllMaps<Gram<true>> mgl;
  AllMaps<Poly<false>> mp;
  AllMaps<Poly<true>> mpl;
  AllMaps<Update<false>> mu;
  // Products of two halves: hi hi, then the second operand's lo (of P X: P's), then the other's.
  const bool few = few_rows(m);
  const int halves = few ? 3 : 1, segs = few ? 3 : p_halves(m) ? 2 : 1, second = 2, third = 4;
  mp.of[0].a[0] = mp.of[0].b[0] = s[0];
  mp.of[0].io[2] = mg.of[0].io[0] = sout[0];
  for (int h = 0; h < 2; ++h) {
    mgl.of[0].io[h] = sout[h];
    mpl.of[0].a[h] = mpl.of[0].b[h] = s[h];
    mpl.of[0].io[2 + h] = sout[h];
    mp.of[0].io[h] = mpl.of[0].io[h] = pout[h];
    (tall ? mu.of[0].b : mu.of[0].a)[h] = p[h];
  }
  for (int i = 0; i < steps; ++i) {
    const float4* factors = st.factors + i;
    const bool last = i + 1 == steps;
    // S = X X^T (X^T X), both operands the same matrix; P from S, which is its own transpose; X's rows times P, or P times X
    for (int h = 0; h < 2; ++h) {
      mg.of[0].a[h] = mg.of[0].b[h] = mgl.of[0].a[h] = mgl.of[0].b[h] = x[i & 1][h];
      (tall ? mu.of[0].a : mu.of[0].b)[h] = x[i & 1][h];
      mu.of[0].io[h] = last ? o : xout[(i + 1) & 1][h];
      mu.of[0].io[2 + h] = xout[i & 1][h];
    }
    const gemm::Args gram = {{{m, m, kx, halves, third, second, tall, tall, 1, n}}, 1, 1, status, 0};
    const gemm::Args poly = {{{m, m, km, halves, third, second, 0, 0, 1, n}}, 1, 1, status, 0};
    ok = few ? run<Gram<true>>(gram, mgl, {}, stream) && run<Poly<true>>(poly, mpl, {at(w.s[0]), at(w.s[1]), w.mpitch, factors, 1}, stream)
             : run<Gram<false>>(gram, mg, {}, stream) &&
                   run<Poly<false>>(poly, mp, {at(w.s[0]), nullptr, w.mpitch, factors, segs > 1}, stream);
    const int p_of = second, x_of = third;
    const gemm::Args upd = {{{rows, cols, km, segs, tall ? x_of : p_of, tall ? p_of : x_of, 0, !tall, 0, n, tall ? 1 : 2}}, 1, 1, status, 0};
    const uint16_t *hi = at(w.x[i & 1][0]), *lo = at(w.x[i & 1][1]);
    ok = ok && (last ? run<Update<true>>(upd, mu, {hi, lo, w.pitch, factors, scale / X_SCALE, out}, stream)
                     : run<Update<false>>(upd, mu, {hi, lo, w.pitch, factors, 1.0f, nullptr}, stream));
    if (!ok) return FLINT_MOE_ECUDA;
  }
  return FLINT_MOE_OK;
}
