// Dense gated feed-forward block on BF16 weights and its gradients (flint_ffn.h), as matrix products of gemm.cuh with
// what stands between them in their epilogues: g and u are columns of one product, whose epilogue makes h of them; dh's
// epilogue makes dg, du and h; dx and the weights' gradients are one launch, since none needs another.
//
// Roundings: h, dg and du enter the next product as bf16, the type of the weights and tokens they are multiplied with (one
// MMA takes one type). h is the rounding point of the expert kernels, so that a dense layer and an expert of the same
// weights agree. Each adds an error of the size of the result's own rounding: the results are within 0.0024 of the exact
// ones in the norm, where rounding once at the end gives 0.0017. Keeping 16 bits as two bf16 halves, as the adapters do
// for their narrow h, would take half as many MMAs again in the forward pass and nearly twice as many in the gradients,
// which the tensor cores bound. All sums are FP32.
//
// 8192 tokens of 2048 x 8192, us a call: forward with g and u kept 555 (1490 TFLOP/s; the first product alone 1650, at
// what the card sustains within its power limit), gradients 1143 (1440; the last four products alone 1750). 77 tokens:
// 33.6, bound by the weights' stream at 3.4 TB/s and two launches' latency.
#include "flint_ffn.h"
#include "gemm.cuh"

namespace flint {
namespace ffn {

using namespace gemm;

// sigmoid(g) and 1 - sigmoid(g), neither as the difference of the other from one. e^-|g| is off by up to 2 + 1.2 |g| steps
// of 2^-23, so that the smaller of the two is.
__device__ __forceinline__ float2 sigmoid2(float g) {
  const float t = __expf(-fabsf(g)), r = __fdividef(1.0f, 1.0f + t);
  return g >= 0.f ? make_float2(r, t * r) : make_float2(t * r, r);
}
// g sigmoid(g): from e^-|g| as well, so that the quotient's divisor lies between one and two. (e^-g itself is too large for
// the fast quotient from g = -87.4 on, and for FP32 from -88.8 on, where g e^g still is a value.)
__device__ __forceinline__ float silu(float g) {
  const float t = __expf(-fabsf(g));
  return __fdividef(g >= 0.f ? g : g * t, 1.0f + t);
}

// bf16 rows [M][N] as they are.
struct Store {
  static constexpr bool PAIR = false, SMALL = false;
  static constexpr int MAPS = MOST, OUTS = 1, INS = 0;
  struct Args {};
  using Pre = NoPre;
  static __device__ __forceinline__ void matrix(const Args&, Part&) {}
  static __device__ __forceinline__ void chunk(const Args&, const MapsOf<Store>& maps, Part& t, int c, uint32_t (&w)[32], uint32_t (&)[32],
                                               const Pre&) {
    const float* v = reinterpret_cast<const float*>(w);
    const uint4 o[4] = {pack8_bf16(v), pack8_bf16(v + 8), pack8_bf16(v + 16), pack8_bf16(v + 24)};
    t.put(&maps.io[0], t.n0 + c, o);
  }
};

// h = silu(g) u from half of the accumulator's columns of g and the same columns of u behind them, and g and u themselves.
template <bool SAVE>
struct Glu {
  static constexpr bool PAIR = true, SMALL = false;
  static constexpr int MAPS = 1, OUTS = 3, INS = 0;
  struct Args {};
  using Pre = NoPre;
  static __device__ __forceinline__ void matrix(const Args&, Part&) {}
  static __device__ __forceinline__ void chunk(const Args&, const MapsOf<Glu>& maps, Part& t, int c, uint32_t (&wg)[32], uint32_t (&wu)[32],
                                               const Pre&) {
    const float* g = reinterpret_cast<const float*>(wg);
    const float* u = reinterpret_cast<const float*>(wu);
    uint4 o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = silu(g[8 * j + i]) * u[8 * j + i];
      o[j] = pack8_bf16(h);
    }
    t.put(&maps.io[0], t.n0 + c, o);
    if (SAVE) {
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = pack8_bf16(g + 8 * j);
      t.put(&maps.io[1], t.n0 + c, o);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = pack8_bf16(u + 8 * j);
      t.put(&maps.io[2], t.n0 + c, o);
    }
  }
};

// dg, du and h from dh and the kept g and u.
struct DGlu {
  static constexpr bool PAIR = false, SMALL = false;
  static constexpr int MAPS = 1, OUTS = 3, INS = 2;
  struct Args {
    const uint16_t* g;  // [M][N]
    const uint16_t* u;
  };
  struct Pre {
    uint4 g[4], u[4];
    __device__ __forceinline__ Pre(const Args& a, const Part& t, int c) {
      const size_t at = (size_t)t.row * t.N + t.n0 + c;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = t.row < t.M && t.n0 + c + 8 * j < t.N;
        g[j] = in ? __ldcg(reinterpret_cast<const uint4*>(a.g + at + 8 * j)) : make_uint4(0, 0, 0, 0);
        u[j] = in ? __ldcg(reinterpret_cast<const uint4*>(a.u + at + 8 * j)) : make_uint4(0, 0, 0, 0);
      }
    }
    __device__ __forceinline__ Pre(const Part& t, const uint8_t* in) {
      slot_row(t, in, g);
      slot_row(t, in + SLOT, u);
    }
  };
  static __device__ __forceinline__ void matrix(const Args&, Part&) {}
  static __device__ __forceinline__ void chunk(const Args&, const MapsOf<DGlu>& maps, Part& t, int c, uint32_t (&w)[32], uint32_t (&)[32],
                                               const Pre& pre) {
    const float* d = reinterpret_cast<const float*>(w);
    uint4 og[4], ou[4], oh[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float g[8], u[8], dg[8], du[8], h[8];
      unpack8_bf16(pre.g[j], g);
      unpack8_bf16(pre.u[j], u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 s = sigmoid2(g[i]);
        const float dh = d[8 * j + i], act = g[i] * s.x;
        dg[i] = dh * u[i] * (s.x * fmaf(g[i], s.y, 1.0f));
        du[i] = dh * act;
        h[i] = act * u[i];
      }
      og[j] = pack8_bf16(dg);
      ou[j] = pack8_bf16(du);
      oh[j] = pack8_bf16(h);
    }
    t.put(&maps.io[0], t.n0 + c, og);
    t.put(&maps.io[1], t.n0 + c, ou);
    t.put(&maps.io[2], t.n0 + c, oh);
  }
};

}  // namespace ffn
}  // namespace flint

using namespace flint;
using namespace flint::ffn;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

flint_moe_status check_shape(const flint_ffn* f) {
  if (!f) return FLINT_MOE_EINVAL;
  if (f->hidden < 8 || f->hidden > 65536 || f->hidden % 8 || f->inter < 8 || f->inter > 65536 || f->inter % 8)
    return FLINT_MOE_EUNSUPPORTED;
  return FLINT_MOE_OK;
}

flint_moe_status check_weights(const flint_ffn* f) {
  const flint_moe_status st = check_shape(f);
  if (st != FLINT_MOE_OK) return st;
  if (!f->gate || !f->up || !f->down) return FLINT_MOE_EINVAL;
  if (!aligned(f->gate, 16) || !aligned(f->up, 16) || !aligned(f->down, 16)) return FLINT_MOE_EALIGN;
  return FLINT_MOE_OK;
}

constexpr int64_t LD_MOST = 0x7fffffff;
bool bad_ld(int64_t ld, int cols) { return ld < cols || ld > LD_MOST; }

// Memory that a call reads or writes; what it writes overlaps nothing else.
struct Span {
  const void* p;
  size_t bytes;
  bool written;
};
size_t rows_bytes(int64_t ld, int cols, int rows) { return rows == 0 ? 0 : 2 * ((size_t)(rows - 1) * ld + cols); }
bool overlap(const Span* s, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < i; ++j) {
      if (!(s[i].written || s[j].written) || !s[i].p || !s[j].p || !s[i].bytes || !s[j].bytes) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(s[i].p), b = reinterpret_cast<uintptr_t>(s[j].p);
      if (a < b + s[j].bytes && b < a + s[i].bytes) return true;
    }
  return false;
}

constexpr int H_STATUS = 1;  // word of the header that flint_moe_read_status reads

struct WsPlan {
  size_t h, dg, du, total;
};
WsPlan ws_plan(const flint_ffn* f, int T, bool grad) {
  WsPlan w = {};
  const size_t act = ws_align((size_t)2 * T * f->inter);
  size_t o = 256;
  w.h = o;
  o += act;
  if (grad) {
    w.dg = o;
    o += act;
    w.du = o;
    o += act;
  }
  w.total = o;
  return w;
}

size_t ws_bytes(const flint_ffn* f, int32_t T, bool grad) {
  if (check_shape(f) != FLINT_MOE_OK || T < 1 || T > FLINT_FFN_MAX_TOKENS) return 0;
  return ws_plan(f, T, grad).total;
}

int blocks_of(int k) { return (k + BK - 1) / BK; }

}  // namespace

extern "C" flint_moe_status flint_ffn_init(int32_t hidden, int32_t inter, const uint16_t* gate, const uint16_t* up,
                                           const uint16_t* down, flint_ffn* out) {
  if (!out) return FLINT_MOE_EINVAL;
  const flint_ffn f = {hidden, inter, gate, up, down};
  const flint_moe_status st = check_weights(&f);
  if (st == FLINT_MOE_OK) *out = f;
  return st;
}

extern "C" size_t flint_ffn_workspace_bytes(const flint_ffn* f, int32_t T) { return ws_bytes(f, T, false); }
extern "C" size_t flint_ffn_backward_workspace_bytes(const flint_ffn* f, int32_t T) { return ws_bytes(f, T, true); }

extern "C" flint_moe_status flint_ffn_forward(const flint_ffn* f, const uint16_t* x, int64_t ldx, int32_t T, uint16_t* y,
                                              int64_t ldy, uint16_t* g, uint16_t* u, void* ws, size_t ws_size,
                                              cudaStream_t stream) {
  flint_moe_status st = check_weights(f);
  if (st != FLINT_MOE_OK) return st;
  if (T < 0 || T > FLINT_FFN_MAX_TOKENS) return FLINT_MOE_EINVAL;
  if (T == 0) return FLINT_MOE_OK;
  const int H = f->hidden, I = f->inter;
  if (!x || !y || !ws || !g != !u || bad_ld(ldx, H) || bad_ld(ldy, H)) return FLINT_MOE_EINVAL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(g, 16) || !aligned(u, 16) || !aligned(ws, 256) || ldx % 8 || ldy % 8)
    return FLINT_MOE_EALIGN;
  const WsPlan w = ws_plan(f, T, false);
  if (ws_size < w.total) return FLINT_MOE_EINVAL;
  const size_t wb = (size_t)2 * H * I, act = (size_t)2 * T * I;
  const Span spans[] = {{f->gate, wb, false}, {f->up, wb, false}, {f->down, wb, false}, {x, rows_bytes(ldx, H, T), false},
                        {y, rows_bytes(ldy, H, T), true}, {g, act, true}, {u, act, true}, {ws, w.total, true}};
  if (overlap(spans, 8)) return FLINT_MOE_EINVAL;
  uint8_t* wsp = static_cast<uint8_t*>(ws);
  uint16_t* h = reinterpret_cast<uint16_t*>(wsp + w.h);
  int* status = reinterpret_cast<int*>(ws) + H_STATUS;
  AllMaps<Glu<true>> m1;
  AllMaps<Store> m2;
  auto& glu = m1.of[0];
  auto& out = m2.of[0];
  bool ok = map_in(&glu.a[0], x, H, T, ldx) && map_in(&glu.b[0], f->gate, H, I, H) && map_in(&glu.b[1], f->up, H, I, H) &&
            map_out(&glu.io[0], h, I, T, I) && map_in(&out.a[0], h, I, T, I) && map_in(&out.b[0], f->down, I, H, I) &&
            map_out(&out.io[0], y, H, T, ldy);
  if (ok && g) ok = map_out(&glu.io[1], g, I, T, I) && map_out(&glu.io[2], u, I, T, I);
  if (!ok) return FLINT_MOE_ECUDA;
  const gemm::Args a1 = {{{T, I, blocks_of(H), 1, 0, 0, 0, 0, 0, 1}}, 1, 0, status, 1};
  const gemm::Args a2 = {{{T, H, blocks_of(I), 1, 0, 0, 0, 0, 0, 1, 2}}, 1, 0, status, 0};
  ok = g ? run<Glu<true>>(a1, m1, {}, stream) : run<Glu<false>>(a1, m1, {}, stream);
  ok = ok && run<Store>(a2, m2, {}, stream);
  return ok ? FLINT_MOE_OK : FLINT_MOE_ECUDA;
}

extern "C" flint_moe_status flint_ffn_backward(const flint_ffn* f, const uint16_t* x, int64_t ldx, const uint16_t* g,
                                               const uint16_t* u, const uint16_t* dy, int64_t lddy, int32_t T, uint16_t* dx,
                                               int64_t lddx, uint16_t* dgate, uint16_t* dup, uint16_t* ddown, void* ws,
                                               size_t ws_size, cudaStream_t stream) {
  flint_moe_status st = check_weights(f);
  if (st != FLINT_MOE_OK) return st;
  if (T < 0 || T > FLINT_FFN_MAX_TOKENS || !dgate != !dup || !dgate != !ddown) return FLINT_MOE_EINVAL;
  const int H = f->hidden, I = f->inter;
  const size_t wb = (size_t)2 * H * I, act = (size_t)2 * T * I;
  if (!aligned(dgate, 16) || !aligned(dup, 16) || !aligned(ddown, 16)) return FLINT_MOE_EALIGN;
  if (T > 0) {
    if (!x || !g || !u || !dy || !ws || bad_ld(ldx, H) || bad_ld(lddy, H) || (dx && bad_ld(lddx, H))) return FLINT_MOE_EINVAL;
    if (!aligned(x, 16) || !aligned(g, 16) || !aligned(u, 16) || !aligned(dy, 16) || !aligned(dx, 16) || !aligned(ws, 256) ||
        ldx % 8 || lddy % 8 || (dx && lddx % 8))
      return FLINT_MOE_EALIGN;
  }
  const WsPlan w = ws_plan(f, T, true);
  if (T > 0 && ws_size < w.total) return FLINT_MOE_EINVAL;
  const Span spans[] = {{f->gate, wb, false}, {f->up, wb, false}, {f->down, wb, false}, {x, rows_bytes(ldx, H, T), false},
                        {g, act, false}, {u, act, false}, {dy, rows_bytes(lddy, H, T), false},
                        {dx, dx ? rows_bytes(lddx, H, T) : 0, true}, {dgate, wb, true}, {dup, wb, true}, {ddown, wb, true},
                        {ws, T > 0 ? w.total : 0, true}};
  if (overlap(spans, 12)) return FLINT_MOE_EINVAL;
  if (T == 0) {
    if (dgate)
      for (uint16_t* p : {dgate, dup, ddown})
        if (cudaMemsetAsync(p, 0, wb, stream) != cudaSuccess) return FLINT_MOE_ECUDA;
    return FLINT_MOE_OK;
  }
  if (!dx && !dgate) return FLINT_MOE_OK;
  uint8_t* wsp = static_cast<uint8_t*>(ws);
  uint16_t *h = reinterpret_cast<uint16_t*>(wsp + w.h), *dg = reinterpret_cast<uint16_t*>(wsp + w.dg),
           *du = reinterpret_cast<uint16_t*>(wsp + w.du);
  int* status = reinterpret_cast<int*>(ws) + H_STATUS;
  CUtensorMap mx, mdy, mg, mu, mgate, mup, mdown, mh, og, ou, oh;
  if (!map_in(&mx, x, H, T, ldx) || !map_in(&mdy, dy, H, T, lddy) || !map_in(&mg, dg, I, T, I) || !map_in(&mu, du, I, T, I) ||
      !map_in(&mgate, f->gate, H, I, H) || !map_in(&mup, f->up, H, I, H) || !map_in(&mdown, f->down, I, H, I) ||
      !map_in(&mh, h, I, T, I) || !map_out(&og, dg, I, T, I) || !map_out(&ou, du, I, T, I) || !map_out(&oh, h, I, T, I))
    return FLINT_MOE_ECUDA;
  AllMaps<DGlu> m1;
  auto& first = m1.of[0];
  first.a[0] = mdy, first.b[0] = mdown, first.io[0] = og, first.io[1] = ou, first.io[2] = oh;
  if (!map_out(&first.io[3], g, I, T, I) || !map_out(&first.io[4], u, I, T, I)) return FLINT_MOE_ECUDA;
  if (!run<DGlu>({{{T, I, blocks_of(H), 1, 0, 0, 0, 1, 0, 1}}, 1, 0, status, 1}, m1, {g, u}, stream)) return FLINT_MOE_ECUDA;
  // dx and the weights' gradients need nothing of one another: one launch, or two where dx has few tiles and many k-blocks
  // (200 tokens of 2048 x 8192: 150 us a call in one). Laid out as if all of them were asked for, so that each has the same
  // bits with and without the others.
  const int kb = blocks_of(T);
  const Problem px = {T, H, blocks_of(I), 2, 2, 2, 0, 1, 0, 1, 2}, pw = {I, H, kb, 1, 0, 0, 1, 1, 0, 1, 2}, pd = {H, I, kb, 1, 0, 0, 1, 1, 0, 1, 1};
  int64_t cycles[3];
  const Choice together = choose<Store>({{px, pw, pw, pd}, 4, 0, nullptr, 0}, &cycles[0]);
  const Choice alone = choose<Store>({{px}, 1, 0, nullptr, 0}, &cycles[1]), rest = choose<Store>({{pw, pw, pd}, 3, 0, nullptr, 0}, &cycles[2]);
  const bool one = cycles[0] <= cycles[1] + cycles[2];
  AllMaps<Store> m2;
  gemm::Args a = {{}, 0, 0, status, 0};
  bool ok = true;
  auto add = [&](const Problem& p, const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b0, const CUtensorMap& b1,
                 uint16_t* out, int64_t ld) {
    MapsOf<Store>& m = m2.of[a.n];
    m.a[0] = a0, m.a[1] = a1, m.b[0] = b0, m.b[1] = b1;
    ok = ok && map_out(&m.io[0], out, p.N, p.M, ld);
    a.p[a.n++] = p;
  };
  if (dx) add(px, mg, mu, mgate, mup, dx, lddx);
  if (dx && !one) {
    if (!ok || !run<Store>(a, m2, {}, stream, alone)) return FLINT_MOE_ECUDA;
    a.n = 0;
  }
  if (dgate) {
    add(pw, mg, mg, mx, mx, dgate, H);
    add(pw, mu, mu, mx, mx, dup, H);
    add(pd, mdy, mdy, mh, mh, ddown, I);
  }
  if (!ok || (a.n > 0 && !run<Store>(a, m2, {}, stream, one ? together : rest))) return FLINT_MOE_ECUDA;
  return FLINT_MOE_OK;
}
