// Low-rank adapters of many requests beside a shared projection, and their
// gradients (C ABI: include/flint_lora.h).
//
// For token t with adapter a (none: nothing is added):
//   h_t = s_a A_a x_t              y_t = bf16(base_t + B_a h_t)
//   g_t = s_a B_a^T dy_t           dx_t = bf16(dx_in_t + A_a^T g_t)
//   dA_a = sum_t g_t x_t^T         dB_a = sum_t dy_t h_t^T
#include <algorithm>

#include "common.cuh"
#include "flint_lora.h"

namespace flint {
namespace lora {

struct Args {
  int K, N, R, n, T;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  const int* adapter;
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* dy;
  int64_t lddy;
  const uint16_t* in;   // y_in or dx_in, bf16, or null
  const float* in32;    // FP32 base [T][N], or null
  uint16_t* out;
  int64_t ldo;
  float* h;  // [T][R]
  float* g;  // [T][R]
  uint16_t* dA;
  uint16_t* dB;
};

__device__ __forceinline__ float b2f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t f2b(float v) {
  const __nv_bfloat16 o = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&o);
}

// One warp per (token, rank): h = s A x, or with GRAD g = s B^T dy.
template <bool GRAD>
__global__ void __launch_bounds__(256) k_lora_shrink(const Args p) {
  const int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (u >= (int64_t)p.T * p.R) return;
  const int t = (int)(u / p.R), r = (int)(u % p.R), a = p.adapter[t];
  float acc = 0.f;
  if (a >= 0 && a < p.n) {
    if (GRAD) {
      for (int n = lane; n < p.N; n += 32) acc += b2f(p.dy[t * p.lddy + n]) * b2f(p.B[((int64_t)a * p.N + n) * p.R + r]);
    } else {
      for (int k = lane; k < p.K; k += 32) acc += b2f(p.x[t * p.ldx + k]) * b2f(p.A[((int64_t)a * p.R + r) * p.K + k]);
    }
    acc *= p.scale[a];
  }
  acc = warp_sum(acc);
  if (lane == 0) (GRAD ? p.g : p.h)[u] = acc;
}

template <bool GRAD>
__global__ void __launch_bounds__(256) k_lora_expand(const Args p) {
  const int D = GRAD ? p.K : p.N;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < (int64_t)p.T * D; u += (int64_t)gridDim.x * 256) {
    const int t = (int)(u / D), c = (int)(u % D), a = p.adapter[t];
    float acc = 0.f;
    if (a >= 0 && a < p.n)
      for (int r = 0; r < p.R; ++r)
        acc += GRAD ? p.g[(int64_t)t * p.R + r] * b2f(p.A[((int64_t)a * p.R + r) * p.K + c])
                    : p.h[(int64_t)t * p.R + r] * b2f(p.B[((int64_t)a * p.N + c) * p.R + r]);
    const float base = p.in32 ? p.in32[u] : (p.in ? b2f(p.in[t * p.ldo + c]) : 0.f);
    p.out[t * p.ldo + c] = f2b(base + acc);
  }
}

// dA (threads over [n][R][K]) and dB (over [n][N][R]).
__global__ void __launch_bounds__(256) k_lora_dw(const Args p) {
  const int64_t na = (int64_t)p.n * p.R * p.K, nb = (int64_t)p.n * p.N * p.R;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < na + nb; u += (int64_t)gridDim.x * 256) {
    float acc = 0.f;
    if (u < na) {
      const int k = (int)(u % p.K), r = (int)(u / p.K % p.R), a = (int)(u / p.K / p.R);
      for (int t = 0; t < p.T; ++t)
        if (p.adapter[t] == a) acc += p.g[(int64_t)t * p.R + r] * b2f(p.x[t * p.ldx + k]);
      p.dA[u] = f2b(acc);
    } else {
      const int64_t v = u - na;
      const int r = (int)(v % p.R), n = (int)(v / p.R % p.N), a = (int)(v / p.R / p.N);
      for (int t = 0; t < p.T; ++t)
        if (p.adapter[t] == a) acc += p.h[(int64_t)t * p.R + r] * b2f(p.dy[t * p.lddy + n]);
      p.dB[v] = f2b(acc);
    }
  }
}

}  // namespace lora
}  // namespace flint

using namespace flint;
using namespace flint::lora;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether two sets of rows (count rows of `cols` bf16, ld apart) share memory, by their extents.
bool overlap(const void* p, int64_t ldp, int colsp, const void* q, int64_t ldq, int colsq, int rows) {
  if (!p || !q || rows == 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  const uintptr_t na = 2 * ((uintptr_t)(rows - 1) * ldp + colsp), nb = 2 * ((uintptr_t)(rows - 1) * ldq + colsq);
  return a < b + nb && b < a + na;
}

flint_moe_status check_lora(const flint_lora* l) {
  if (!l) return FLINT_MOE_EINVAL;
  if (l->in_dim < 8 || l->in_dim > 65536 || l->in_dim % 8 || l->out_dim < 8 || l->out_dim > 65536 || l->out_dim % 8)
    return FLINT_MOE_EUNSUPPORTED;
  if (l->rank < 8 || l->rank > FLINT_LORA_MAX_RANK || l->rank % 8) return FLINT_MOE_EUNSUPPORTED;
  if (l->num_adapters < 1 || l->num_adapters > FLINT_LORA_MAX_ADAPTERS) return FLINT_MOE_EUNSUPPORTED;
  return FLINT_MOE_OK;
}

flint_moe_status check_pool(const flint_lora* l) {
  const flint_moe_status st = check_lora(l);
  if (st != FLINT_MOE_OK) return st;
  if (!l->a || !l->b || !l->scale) return FLINT_MOE_EINVAL;
  if (!aligned(l->a, 16) || !aligned(l->b, 16) || !aligned(l->scale, 4)) return FLINT_MOE_EALIGN;
  return FLINT_MOE_OK;
}

struct WsPlan {
  size_t h, g, y32, total;
};
WsPlan ws_plan(const flint_lora* l, int T, bool grad, bool base) {
  WsPlan w;
  size_t o = 0;
  w.h = o;    o = ws_align(o + sizeof(float) * (size_t)T * l->rank);
  w.g = o;    o = ws_align(o + (grad ? sizeof(float) * (size_t)T * l->rank : 0));
  w.y32 = o;  o = ws_align(o + (base ? sizeof(float) * (size_t)T * l->out_dim : 0));
  w.total = o;
  return w;
}

Args make_args(const flint_lora* l, const int32_t* adapter, int T) {
  Args p = {};
  p.K = l->in_dim;
  p.N = l->out_dim;
  p.R = l->rank;
  p.n = l->num_adapters;
  p.T = T;
  p.A = l->a;
  p.B = l->b;
  p.scale = l->scale;
  p.adapter = adapter;
  return p;
}

int blocks(int64_t threads) { return (int)std::min<int64_t>(152 * 16, (threads + 255) / 256); }

}  // namespace

extern "C" flint_moe_status flint_lora_init(int32_t in_dim, int32_t out_dim, int32_t rank, int32_t num_adapters,
                                            const uint16_t* a, const uint16_t* b, const float* scale, flint_lora* out) {
  if (!out) return FLINT_MOE_EINVAL;
  const flint_lora l = {in_dim, out_dim, rank, num_adapters, a, b, scale};
  const flint_moe_status st = check_pool(&l);
  if (st == FLINT_MOE_OK) *out = l;
  return st;
}

extern "C" size_t flint_lora_workspace_bytes(const flint_lora* l, int32_t max_tokens) {
  if (check_lora(l) != FLINT_MOE_OK || max_tokens < 1 || max_tokens > FLINT_LORA_MAX_TOKENS) return 0;
  return ws_plan(l, max_tokens, false, false).total;
}

extern "C" size_t flint_gemv_lora_workspace_bytes(const flint_lora* l, int32_t max_batch) {
  if (check_lora(l) != FLINT_MOE_OK || max_batch < 1 || max_batch > MAX_BATCH) return 0;
  return ws_plan(l, max_batch, false, true).total;
}

extern "C" size_t flint_lora_backward_workspace_bytes(const flint_lora* l, int32_t max_tokens) {
  if (check_lora(l) != FLINT_MOE_OK || max_tokens < 1 || max_tokens > FLINT_LORA_MAX_TOKENS) return 0;
  return ws_plan(l, max_tokens, true, false).total;
}

extern "C" flint_moe_status flint_lora_apply(const flint_lora* l, const uint16_t* x, int64_t ldx, const int32_t* adapter,
                                             int32_t T, const uint16_t* y_in, uint16_t* y_out, int64_t ldy, void* ws,
                                             size_t ws_bytes, cudaStream_t stream) {
  const flint_moe_status st = check_pool(l);
  if (st != FLINT_MOE_OK) return st;
  if (T < 0 || T > FLINT_LORA_MAX_TOKENS || ldx < l->in_dim || ldy < l->out_dim) return FLINT_MOE_EINVAL;
  if (T == 0) return FLINT_MOE_OK;
  if (!x || !adapter || !y_out || !ws) return FLINT_MOE_EINVAL;
  if (!aligned(x, 16) || !aligned(y_in, 16) || !aligned(y_out, 16) || !aligned(ws, 256) || !aligned(adapter, 4) || ldx % 8 ||
      ldy % 8)
    return FLINT_MOE_EALIGN;
  if (overlap(y_out, ldy, l->out_dim, x, ldx, l->in_dim, T) ||
      (y_in != y_out && overlap(y_out, ldy, l->out_dim, y_in, ldy, l->out_dim, T)))
    return FLINT_MOE_EINVAL;
  const WsPlan w = ws_plan(l, T, false, false);
  if (ws_bytes < w.total) return FLINT_MOE_EINVAL;
  Args p = make_args(l, adapter, T);
  p.x = x;
  p.ldx = ldx;
  p.in = y_in;
  p.out = y_out;
  p.ldo = ldy;
  p.h = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.h);
  k_lora_shrink<false><<<(int)(((int64_t)T * p.R + 7) / 8), 256, 0, stream>>>(p);
  k_lora_expand<false><<<blocks((int64_t)T * p.N), 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FLINT_MOE_OK : FLINT_MOE_ECUDA;
}

extern "C" flint_moe_status flint_gemv_lora(const void* packed, int32_t N, int32_t K, int32_t fmt, const uint16_t* x,
                                            int32_t B, uint16_t* y, const flint_lora* l, const int32_t* adapter, void* ws,
                                            size_t ws_bytes, int32_t* dev_status, cudaStream_t stream) {
  flint_moe_status st = check_pool(l);
  if (st != FLINT_MOE_OK) return st;
  if (flint_gemv_packed_bytes(N, K, fmt) == 0) return FLINT_MOE_EUNSUPPORTED;
  if (B < 0 || B > MAX_BATCH || l->in_dim != K || l->out_dim != N) return FLINT_MOE_EINVAL;
  if (B == 0) return FLINT_MOE_OK;
  if (!packed || !x || !y || !adapter || !ws) return FLINT_MOE_EINVAL;
  if (!aligned(ws, 256) || !aligned(adapter, 4) || !aligned(dev_status, 4)) return FLINT_MOE_EALIGN;
  if (overlap(y, N, N, x, K, K, B)) return FLINT_MOE_EINVAL;
  const WsPlan w = ws_plan(l, B, false, true);
  if (ws_bytes < w.total) return FLINT_MOE_EINVAL;
  Args p = make_args(l, adapter, B);
  p.x = x;
  p.ldx = K;
  float* y32 = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.y32);
  p.in32 = y32;
  p.out = y;
  p.ldo = N;
  p.h = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.h);
  st = gemv_impl(packed, N, K, fmt, x, B, y, y32, nullptr, 0.f, dev_status, stream);
  if (st != FLINT_MOE_OK) return st;
  k_lora_shrink<false><<<(int)(((int64_t)B * p.R + 7) / 8), 256, 0, stream>>>(p);
  k_lora_expand<false><<<blocks((int64_t)B * p.N), 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FLINT_MOE_OK : FLINT_MOE_ECUDA;
}

extern "C" flint_moe_status flint_lora_backward(const flint_lora* l, const uint16_t* x, int64_t ldx, const uint16_t* dy,
                                                int64_t lddy, const int32_t* adapter, int32_t T, const uint16_t* dx_in,
                                                uint16_t* dx_out, int64_t lddx, uint16_t* da, uint16_t* db, void* ws,
                                                size_t ws_bytes, cudaStream_t stream) {
  const flint_moe_status st = check_pool(l);
  if (st != FLINT_MOE_OK) return st;
  if (T < 0 || T > FLINT_LORA_MAX_TOKENS || ldx < l->in_dim || lddy < l->out_dim || (dx_out && lddx < l->in_dim))
    return FLINT_MOE_EINVAL;
  if (!da || !db) return FLINT_MOE_EINVAL;
  if (!aligned(da, 16) || !aligned(db, 16)) return FLINT_MOE_EALIGN;
  const size_t nw = (size_t)l->num_adapters * l->rank;
  if (T == 0) {
    if (cudaMemsetAsync(da, 0, nw * l->in_dim * 2, stream) != cudaSuccess ||
        cudaMemsetAsync(db, 0, nw * l->out_dim * 2, stream) != cudaSuccess)
      return FLINT_MOE_ECUDA;
    return FLINT_MOE_OK;
  }
  if (!x || !dy || !adapter || !ws) return FLINT_MOE_EINVAL;
  if (!aligned(x, 16) || !aligned(dy, 16) || !aligned(dx_in, 16) || !aligned(dx_out, 16) || !aligned(ws, 256) ||
      !aligned(adapter, 4) || ldx % 8 || lddy % 8 || (dx_out && lddx % 8))
    return FLINT_MOE_EALIGN;
  if (dx_out && (overlap(dx_out, lddx, l->in_dim, x, ldx, l->in_dim, T) ||
                 overlap(dx_out, lddx, l->in_dim, dy, lddy, l->out_dim, T) ||
                 (dx_in != dx_out && overlap(dx_out, lddx, l->in_dim, dx_in, lddx, l->in_dim, T))))
    return FLINT_MOE_EINVAL;
  const WsPlan w = ws_plan(l, T, true, false);
  if (ws_bytes < w.total) return FLINT_MOE_EINVAL;
  Args p = make_args(l, adapter, T);
  p.x = x;
  p.ldx = ldx;
  p.dy = dy;
  p.lddy = lddy;
  p.in = dx_in;
  p.out = dx_out;
  p.ldo = lddx;
  p.h = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.h);
  p.g = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.g);
  p.dA = da;
  p.dB = db;
  const int sg = (int)(((int64_t)T * p.R + 7) / 8);
  k_lora_shrink<false><<<sg, 256, 0, stream>>>(p);
  k_lora_shrink<true><<<sg, 256, 0, stream>>>(p);
  if (dx_out) k_lora_expand<true><<<blocks((int64_t)T * p.K), 256, 0, stream>>>(p);
  k_lora_dw<<<blocks((int64_t)nw * (p.K + p.N)), 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FLINT_MOE_OK : FLINT_MOE_ECUDA;
}
