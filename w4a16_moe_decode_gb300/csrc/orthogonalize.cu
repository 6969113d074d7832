// Orthogonalised updates by Newton-Schulz steps (flint_orthogonalize.h), as matrix products of gemm.cuh.
//
// Scaled values: X is kept times 2^10 as hi + lo (f16), S times 2^10 and P times 2^8 (f16).
#include <cmath>

#include "flint_orthogonalize.h"
#include "gemm.cuh"

namespace flint {
namespace ortho {

using namespace gemm;

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
// X = M / (|M| + eps): the sums of squares in FP64 (a block's partial sum each),
// then hi and lo. Eight values share a power of two, so that squares neither
// overflow nor vanish.
// ---------------------------------------------------------------------------
struct Start {
  const void* in;
  int bf16, n, rows, cols, pitch, parts;
  float eps;
  double* part;  // [n][parts]
  uint16_t *hi, *lo;
  int* status;
};

constexpr int START_THREADS = 256;

__device__ __forceinline__ float load1(const Start& a, size_t i) {
  return a.bf16 ? bf16lo(static_cast<const uint16_t*>(a.in)[i]) : static_cast<const float*>(a.in)[i];
}
// Values i .. i + 7 (i a multiple of 8 from an aligned start).
__device__ __forceinline__ void load8(const Start& a, size_t i, float* v) {
  if (a.bf16) {
    unpack8_bf16(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.in) + i), v);
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.in) + i);
    const float4 x = p[0], y = p[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  }
}

__global__ void __launch_bounds__(START_THREADS) k_ortho_norm(const Start a) {
  __shared__ double s_sum[START_THREADS / 32];
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0 && blockIdx.x + blockIdx.y == 0) *a.status = 0;
  const size_t all = (size_t)a.rows * a.cols, first = blockIdx.y * all;
  const bool vec = all % 8 == 0;
  double sum = 0.0;
  for (size_t i = 8 * ((size_t)blockIdx.x * START_THREADS + threadIdx.x); i < all; i += (size_t)gridDim.x * START_THREADS * 8) {
    float v[8];
    if (vec) {
      load8(a, first + i, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = i + e < all ? load1(a, first + i + e) : 0.f;
    }
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]));
    const int ex = min(max((int)(__float_as_uint(mx) >> 23) - 127, -126), 126);
    const float sc = exp2i(-ex);
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(v[e] * sc, v[e] * sc, q);
    sum = fma((double)q, __longlong_as_double((long long)(1023 + 2 * ex) << 52), sum);
  }
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
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 32) {
    double sum = 0.0;
    for (int p = threadIdx.x; p < a.parts; p += 32) sum += __ldcg(a.part + (size_t)blockIdx.y * a.parts + p);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (threadIdx.x == 0) {  // 1 / (|M| + eps) as two FP32 factors, since a large norm's is below FP32's normals
      const double d = sqrt(sum) + (double)a.eps;
      const int half = ((int)(__double_as_longlong(d) >> 52) - 1023) / 2;
      s_scale[0] = exp2i(-half);
      s_scale[1] = (float)(X_SCALE / (d * __longlong_as_double((long long)(1023 - half) << 52)));
    }
  }
  __syncthreads();
  const float s0 = s_scale[0], s1 = s_scale[1];
  const size_t all = (size_t)a.rows * a.cols, first = blockIdx.y * all, out = (size_t)blockIdx.y * a.rows * a.pitch;
  const size_t step = (size_t)gridDim.x * START_THREADS;
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
    for (size_t i = (size_t)blockIdx.x * START_THREADS + threadIdx.x; i < all; i += step) {
      const size_t r = i / a.cols, at = out + r * a.pitch + (i - r * a.cols);
      const float v = (load1(a, first + i) * s0) * s1;
      const __half h = __float2half_rn(v);
      a.hi[at] = *reinterpret_cast<const uint16_t*>(&h);
      const __half l = __float2half_rn(v - __half2float(h));
      a.lo[at] = *reinterpret_cast<const uint16_t*>(&l);
    }
  }
}

// ---------------------------------------------------------------------------
// Epilogues: S, P = b S + c S S, X <- a X + P X.
// ---------------------------------------------------------------------------
struct Gram {
  static constexpr bool PAIR = false;
  static constexpr int MAPS = 1;
  struct Args {};
  struct Pre {
    __device__ __forceinline__ Pre(const Args&, const Part&, int) {}
  };
  static __device__ __forceinline__ void chunk(const Args&, const Maps& maps, Part& t, int c, uint32_t (&w)[32], uint32_t (&)[32],
                                               const Pre&) {
    float* v = reinterpret_cast<float*>(w);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= S_SCALE / (X_SCALE * X_SCALE);
    const uint4 o[4] = {pack8_f16(v), pack8_f16(v + 8), pack8_f16(v + 16), pack8_f16(v + 24)};
    t.put(&maps.out[0], t.n0 + c, o);
    if (t.twice) t.put_transposed(&maps.out[0], t.n0 + c, o);
  }
};

// 32 columns of this lane's row of a matrix [batch][M][pitch], from the tile's column c on; zero outside.
__device__ __forceinline__ void load_row(const Part& t, const uint16_t* m, int pitch, int c, uint4 (&v)[4]) {
  const uint16_t* at = m + ((size_t)t.z * t.M + t.row) * pitch + t.n0 + c;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = t.row < t.M && t.n0 + c + 8 * j < t.N ? __ldcg(reinterpret_cast<const uint4*>(at + 8 * j)) : make_uint4(0, 0, 0, 0);
}

struct Poly {
  static constexpr bool PAIR = false;
  static constexpr int MAPS = 1;
  struct Args {
    const uint16_t* s;
    int pitch;
    float b, c;
    int lo;  // P's second half too
  };
  struct Pre {
    uint4 s[4];
    __device__ __forceinline__ Pre(const Args& a, const Part& t, int c) { load_row(t, a.s, a.pitch, c, s); }
  };
  static __device__ __forceinline__ void chunk(const Args& a, const Maps& maps, Part& t, int c, uint32_t (&w)[32], uint32_t (&)[32],
                                               const Pre& pre) {
    const float fs = a.b * (P_SCALE / S_SCALE), fq = a.c * (P_SCALE / (S_SCALE * S_SCALE));
    uint4 hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[8];
      unpack8_f16(pre.s[j], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(fs, v[i], fq * __uint_as_float(w[8 * j + i]));
      split8(v, hi[j], lo[j]);
    }
    t.put(&maps.out[0], t.n0 + c, hi);
    if (t.twice) t.put_transposed(&maps.out[0], t.n0 + c, hi);
    if (a.lo) {
      t.put(&maps.out[1], t.n0 + c, lo);
      if (t.twice) t.put_transposed(&maps.out[1], t.n0 + c, lo);
    }
  }
};

template <bool LAST>
struct Update {
  static constexpr bool PAIR = false;
  static constexpr int MAPS = 1;
  struct Args {
    const uint16_t *hi, *lo;
    int pitch;
    float a, scale;
    uint16_t* out;  // LAST: [batch][M][N]
  };
  struct Pre {
    uint4 hi[4], lo[4];
    __device__ __forceinline__ Pre(const Args& a, const Part& t, int c) {
      load_row(t, a.hi, a.pitch, c, hi);
      load_row(t, a.lo, a.pitch, c, lo);
    }
  };
  static __device__ __forceinline__ void chunk(const Args& a, const Maps& maps, Part& t, int c, uint32_t (&w)[32], uint32_t (&)[32],
                                               const Pre& pre) {
    constexpr float fp = 1.0f / P_SCALE;  // P X comes scaled by both
    uint4 hv[4], lv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float h[8], l[8], v[8];
      unpack8_f16(pre.hi[j], h);
      unpack8_f16(pre.lo[j], l);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(fp, __uint_as_float(w[8 * j + i]), a.a * (h[i] + l[i]));
      if (LAST) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= a.scale;
        hv[j] = pack8_bf16(v);
      } else {
        split8(v, hv[j], lv[j]);
      }
    }
    if (!LAST || t.N % 8 == 0) {
      t.put(&maps.out[0], t.n0 + c, hv);
      if (!LAST) t.put(&maps.out[1], t.n0 + c, lv);
    } else {  // rows that TMA cannot reach: through a slot, a row's neighbours by neighbouring lanes
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) *t.piece(0, j) = hv[j];
      __syncwarp();
      const int col = t.n0 + c + t.lane;
      for (int r = 0; r < 32 && t.row0 + r < t.M; ++r)
        if (col < t.N)
          a.out[((size_t)t.z * t.M + t.row0 + r) * t.N + col] =
              *reinterpret_cast<const uint16_t*>(t.sm + r * 64 + ((((t.lane >> 3) ^ (r >> 1)) & 3) << 4) + (t.lane & 7) * 2);
    }
  }
};

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

// Blocks of a matrix in the first two kernels: eight pieces of eight values a thread, 128 at most.
int parts_of(int rows, int cols) {
  const int64_t per = 8 * 8 * START_THREADS;
  return (int)std::min<int64_t>(128, ((int64_t)rows * cols + per - 1) / per);
}

// P X as P_hi X_hi + P_lo X_hi + P_hi X_lo up to this many rows, where the products are cheap beside X's traffic and few
// rounding errors meet in a result; above, as P_hi X_hi, whose errors average out.
bool few_rows(int m) { return m <= 128; }

struct WsPlan {
  int m, pitch, mpitch, parts;
  size_t part, x[2][2], s, p[2], total;  // x: of even and odd steps; x, p: hi and lo
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
  for (int i = 0; i < 4; ++i) {
    w.x[i >> 1][i & 1] = o;
    o += xb;
  }
  w.s = o;
  o += mb;
  for (int i = 0; i < 2; ++i) {
    w.p[i] = o;
    o += i == 0 || few_rows(w.m) ? mb : 0;
  }
  w.total = o;
  return w;
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
  uint8_t* wsp = static_cast<uint8_t*>(ws);
  int* status = reinterpret_cast<int*>(ws) + H_STATUS;
  auto at = [&](size_t o) { return reinterpret_cast<uint16_t*>(wsp + o); };
  const bool tall = rows > cols;
  const int m = w.m;
  CUtensorMap x[2][2], xout[2][2], s, sout, p[2], pout[2], o;
  auto map = [&](CUtensorMap* mp, size_t off, int64_t c, int64_t r, int64_t pitch, bool as_out) {
    return map_matrix(mp, at(off), c, r, pitch, n, r * pitch, as_out);
  };
  bool ok = map(&s, w.s, m, m, w.mpitch, false) && map(&sout, w.s, m, m, w.mpitch, true);
  for (int i = 0; i < 2; ++i) {
    for (int h = 0; h < 2; ++h)
      ok = ok && map(&x[i][h], w.x[i][h], cols, rows, w.pitch, false) && map(&xout[i][h], w.x[i][h], cols, rows, w.pitch, true);
    ok = ok && map(&p[i], w.p[i], m, m, w.mpitch, false) && map(&pout[i], w.p[i], m, m, w.mpitch, true);
  }
  o = sout;
  if (cols % 8 == 0) ok = ok && map_matrix(&o, out, cols, rows, cols, n, (int64_t)rows * cols, true);
  if (!ok) return FLINT_MOE_ECUDA;
  const Start st = {in, fmt == FLINT_ORTHOGONALIZE_BF16, n, rows, cols, w.pitch, w.parts, eps,
                    reinterpret_cast<double*>(wsp + w.part), at(w.x[0][0]), at(w.x[0][1]), status};
  const dim3 grid((unsigned)w.parts, (unsigned)n);
  if (!launch<k_ortho_norm>(grid, START_THREADS, 0, 0, stream, st) || !launch<k_ortho_split>(grid, START_THREADS, 0, 0, stream, st))
    return FLINT_MOE_ECUDA;
  const int kx = ((tall ? rows : cols) + BK - 1) / BK, km = (m + BK - 1) / BK;
  AllMaps<1> mg, mp, mu;
  mp.of[0].a[0] = mp.of[0].b[0] = s;
  mg.of[0].out[0] = sout;
  const bool few = few_rows(m);
  for (int h = 0; h < 2; ++h) {
    mp.of[0].out[h] = pout[h];
    (tall ? mu.of[0].b : mu.of[0].a)[h] = p[h];
  }
  for (int i = 0; i < steps; ++i) {
    const float* cf = coeffs + 3 * i;
    const bool last = i + 1 == steps;
    // S = X X^T (X^T X), both operands the same matrix; P from S, which is its own transpose; X's rows times P, or P times X
    mg.of[0].a[0] = mg.of[0].b[0] = x[i & 1][0];
    for (int h = 0; h < 2; ++h) {
      (tall ? mu.of[0].a : mu.of[0].b)[h] = x[i & 1][h];
      mu.of[0].out[h] = last ? o : xout[(i + 1) & 1][h];
    }
    ok = run<Gram>({{{m, m, kx, 1, 0, 0, tall, tall, 1, n}}, 1, 1, status, 0}, mg, {}, stream) &&
         run<Poly>({{{m, m, km, 1, 0, 0, 0, 0, 1, n}}, 1, 1, status, 0}, mp, {at(w.s), w.mpitch, cf[1], cf[2], few}, stream);
    const int p_of = 2, x_of = 4;  // hi hi, then P_lo, then X_lo
    const gemm::Args upd = {{{rows, cols, km, few ? 3 : 1, tall ? x_of : p_of, tall ? p_of : x_of, 0, !tall, 0, n}}, 1, 1, status, 0};
    const uint16_t *hi = at(w.x[i & 1][0]), *lo = at(w.x[i & 1][1]);
    ok = ok && (last ? run<Update<true>>(upd, mu, {hi, lo, w.pitch, cf[0], scale / X_SCALE, out}, stream)
                     : run<Update<false>>(upd, mu, {hi, lo, w.pitch, cf[0], 1.0f, nullptr}, stream));
    if (!ok) return FLINT_MOE_ECUDA;
  }
  return FLINT_MOE_OK;
}
