// Low-rank adapters of many requests beside a shared projection, and their
// gradients (C ABI: include/flint_lora.h).
//
// For token t with adapter a (none: nothing is added):
//   h_t = s_a A_a x_t              y_t = bf16(base_t + B_a h_t)
//   g_t = s_a B_a^T dy_t           dx_t = bf16(dx_in_t + A_a^T g_t)
//   dA_a = sum_t g_t x_t^T         dB_a = sum_t dy_t h_t^T
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "flint_lora.h"
#include "tensor.cuh"

namespace flint {
namespace lora {

constexpr int TM = 128;       // tokens of a tile (the tensor cores' M)
constexpr int BK = 64;        // columns of one 128-byte swizzled row
constexpr int BOX = TM * BK * 2;   // 16 KiB: 128 rows x 64 columns
constexpr int HALF = BOX / 2;      // 8 KiB: 64 rows x 64 columns
enum : int { H_STATUS = HDR_STATUS, H_TILES = 2, H_CHUNKS = 3 };

// A tile: up to 128 tokens of one adapter (-1: tokens without one). Its row r is
// token rowmap[tile * 128 + r]; rows past `count` repeat the last token there, so
// that every row can be loaded, and are zero in h and g.
struct Args {
  int K, N, R, Rp, n, T;  // Rp: R rounded up to 16, the tensor cores' step
  const float* scale;
  const int* adapter;
  int with_none;  // tokens without an adapter get tiles (their output rows have to be written)
  int max_tiles;
  int* hdr;
  int2* tiles;   // [max_tiles]: {adapter, count}, {-2, 0} past the last
  int* rowmap;   // [max_tiles * 128]
  uint16_t* h;   // s A x as bf16 halves hi, lo: [2][max_tiles * 128][R]
  uint16_t* g;   // s B^T dy likewise
  const uint16_t* x;
  const uint16_t* dy;
  const uint16_t* in;  // y_in or dx_in, or null
  uint16_t* out;
  int ldx, lddy, ldo;  // row strides in elements (offsets of rows are 64-bit products)
  // weights' gradients
  int CT;              // tiles of a chunk at most
  int slabs_a, slabs_b;  // 128-wide slabs of K and of N
  int4* chunks;        // {adapter, first tile, tiles, partial slot or -1}
  int2* of_adapter;    // {first partial slot, chunks} of each adapter
  float* part;         // [slot][R K + N R]
  uint16_t* dA;
  uint16_t* dB;
};

struct Maps {
  CUtensorMap a;     // A [n][R][K]: boxes 64 x Rp
  CUtensorMap b;     // B [n][N][R]: boxes 64 x 64
  CUtensorMap h, g;  // [2 * max_tiles * 128][R], boxes 64 x 64
  // Token rows, for runs of neighbouring tokens: boxes of 64 columns x 32 rows (shrink) and x 16 (gradients), and
  // of 32 columns x 32 rows in the 64-byte swizzle (base and output rows)
  CUtensorMap x32, dy32, x16, dy16, in, out;
};

__device__ __forceinline__ uint16_t f2b(float v) {
  const __nv_bfloat16 o = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&o);
}
__device__ __forceinline__ uint32_t f2b2(float lo, float hi) {
  const __nv_bfloat162 o = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&o);
}

// Four values of h or g as bf16 halves: hi + lo carries 16 significant bits of the FP32 sum into the next product,
// whose operands are bf16 on the tensor cores; a third half would carry 24, for half as many MMAs again and half as
// much more of h in memory, and change an output by 2^-16 of a term where its own rounding changes it by 2^-8.
// hi stops at bf16's largest: of a finite value beyond it lo holds the rest, of an infinity lo is infinite.
__device__ __forceinline__ uint32_t f2b2_finite(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void halves(const float4 v, uint2& hi, uint2& lo) {
  hi = make_uint2(f2b2_finite(v.x, v.y), f2b2_finite(v.z, v.w));
  lo = make_uint2(f2b2(v.x - bf16lo(hi.x), v.y - bf16hi(hi.x)), f2b2(v.z - bf16lo(hi.y), v.w - bf16hi(hi.y)));
}

// ---------------------------------------------------------------------------
// Plan (one block): tokens sorted by adapter, stably, into tiles. Warp w owns a
// run of consecutive tokens; the 32 tokens of a step find their fellows with
// match_any, so every token's place follows from counts and lane masks alone.
// Short loops on purpose: between calls that stream 100 MB the code itself comes
// from memory, and every stretch of it costs up to a microsecond. Bound by that
// and by the chain of its barriers: 7.8 us alone and cold for 8192 tokens.
// ---------------------------------------------------------------------------
constexpr int PLAN_T = 16384;  // tokens whose adapters fit in shared memory beside the counts
__host__ __device__ inline size_t plan_smem(int n, int T) {
  return sizeof(int) * ((size_t)34 * (n + 1) + 3 * (n + 2) + (T <= PLAN_T ? T : 0));
}

// Exclusive sums of f(0 .. n-1) into out[0 .. n], by one warp, 32 at a time.
template <typename F>
__device__ __forceinline__ void warp_scan(int n, int lane, int* out, F f) {
  int carry = 0;
#pragma unroll 1
  for (int base = 0; base < n; base += 32) {
    const int i = base + lane, v = i < n ? f(i) : 0;
    int inc = v;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (i < n) out[i] = carry + inc - v;
    carry += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) out[n] = carry;
}

// The last g in [0, n) with first[g] <= i: the group of item i < first[n].
__device__ __forceinline__ int group_of(const int* first, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (first[m] <= i)
      lo = m;
    else
      hi = m;
  }
  return lo;
}

__global__ void __launch_bounds__(1024) k_lora_plan(const Args a) {
  extern __shared__ int sm[];
  const int G = a.n + 1;  // group n: tokens without an adapter
  int* hist = sm;         // [32][G], then each warp's next place in the group
  int* cnt = hist + 32 * G;
  int* lasts = cnt + G;    // last token of each group
  int* tf = lasts + G;     // first tile of each group
  int* cf = tf + G + 1;    // first chunk
  int* sf = cf + G + 1;    // first partial slot
  int* ids = sf + G + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < 32 * G; i += 1024) hist[i] = 0;
  pdl_wait();
  pdl_trigger();
  // The tokens' adapters in shared memory, all asked for at once; past PLAN_T of them they stay where they are.
  const bool staged = a.T <= PLAN_T;
  if (staged) {
#pragma unroll 4
    for (int i = threadIdx.x; i < a.T; i += 1024) ids[i] = __ldg(a.adapter + i);
  }
  __syncthreads();
  const int* src = staged ? ids : a.adapter;
  const int L = (a.T + 1023) / 1024 * 32, t0 = warp * L, t1 = min(a.T, t0 + L);
  int* mine = hist + warp * G;
  // One step of 32 tokens from i: the group of this lane's (-1: none) and its place behind what mine[] holds, which
  // then grows by the step's tokens.
  auto step = [&](int i, int& g) {
    g = -1;
    if (i + lane < t1) {
      g = src[i + lane];
      if (g < 0 || g >= a.n) g = a.n;
    }
    const unsigned same = __match_any_sync(0xffffffffu, g);
    const int rank = __popc(same & ((1u << lane) - 1));
    int at = 0;
    if (g >= 0) at = mine[g] + rank;
    __syncwarp();
    if (g >= 0 && rank == 0) mine[g] += __popc(same);
    __syncwarp();
    return at;
  };
#pragma unroll 1
  for (int i = t0; i < t1; i += 32) {
    int g;
    step(i, g);
  }
  __syncthreads();
  for (int c = warp; c < G; c += 32) {  // the warps' counts of a group -> their first places in it
    const int v = hist[lane * G + c];
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    hist[lane * G + c] = inc - v;
    if (lane == 31) cnt[c] = c == a.n && !a.with_none ? 0 : inc;
  }
  __syncthreads();
  auto tiles_of = [&](int c) { return (cnt[c] + TM - 1) / TM; };
  auto chunks_of = [&](int c) { return c == a.n ? 0 : (tiles_of(c) + a.CT - 1) / a.CT; };
  // warps 0 .. 2: the first tile, chunk and partial slot of each group
  if (warp < (a.chunks ? 3 : 1))
    warp_scan(G, lane, warp == 0 ? tf : warp == 1 ? cf : sf, [&](int c) {
      if (warp == 0) return tiles_of(c);
      const int k = chunks_of(c);
      return warp == 2 && k == 1 ? 0 : k;
    });
  __syncthreads();
#pragma unroll 1
  for (int i = t0; i < t1; i += 32) {
    int g;
    const int at = step(i, g);
    if (g >= 0 && at < cnt[g]) {  // (no place for tokens without an adapter where they need none)
      a.rowmap[tf[g] * TM + at] = i + lane;
      if (at == cnt[g] - 1) lasts[g] = i + lane;
    }
  }
  __syncthreads();
  const int ntiles = tf[G];
  for (int i = threadIdx.x; i < a.max_tiles; i += 1024) {
    int2 tile = make_int2(-2, 0);  // no tile
    if (i < ntiles) {
      const int c = group_of(tf, G, i);
      tile = make_int2(c == a.n ? -1 : c, min(TM, cnt[c] - TM * (i - tf[c])));
    }
    a.tiles[i] = tile;
  }
  for (int c = warp; c < G; c += 32) {  // rows past the count of a group's last tile repeat its last token
    const int end = tf[c + 1] * TM;
    for (int r = tf[c] * TM + cnt[c] + lane; r < end; r += 32) a.rowmap[r] = lasts[c];
  }
  if (a.chunks) {
    const int nchunks = cf[G];
    for (int i = threadIdx.x; i < nchunks; i += 1024) {
      const int c = group_of(cf, G, i), j = i - cf[c];
      a.chunks[i] = make_int4(c, tf[c] + j * a.CT, min(a.CT, tiles_of(c) - j * a.CT), chunks_of(c) > 1 ? sf[c] + j : -1);
    }
    for (int c = threadIdx.x; c < a.n; c += 1024) a.of_adapter[c] = make_int2(sf[c], chunks_of(c));
    if (threadIdx.x == 0) a.hdr[H_CHUNKS] = nchunks;
  }
  if (threadIdx.x == 0) {
    a.hdr[H_STATUS] = 0;
    a.hdr[H_TILES] = ntiles;
  }
}

// ---------------------------------------------------------------------------
// Token rows: a warp whose rows are neighbouring tokens (a request's prompt) moves them with one TMA box; others,
// in any order, are gathered with 16-byte asynchronous copies that arrive on the stage's mbarrier by themselves.
// (TMA's four-row gather delivered one such group every 50 to 60 ns and SM, 1.2 TB/s over the card, whatever the
// order; base and output rows by 16-byte copies and stores only took 69 us for 8192 tokens of 2048 x 8192.)
//
// Shrink: h = s A x of one tile (z = 0) or g = s B^T dy (z = 1), [128 x D] times
// [D x R] on the tensor cores. A cluster of S CTAs shares a tile; CTA s takes a
// run of the 64-column k-blocks, and the partial sums meet in distributed shared
// memory, added in CTA order. Bound by the token rows it reads: per k-block 16 KiB
// of them against at most 16 KiB of weights from L2. 14.4 us alone and cold for
// 8192 tokens of 2048, rank 64 (34 MB: 2.4 TB/s; the start, the sums and the one
// wave of two CTAs an SM leave half of it to the copies).
//   warps 0-3  token rows into the stages; later the accumulator, tensor memory
//              -> shared memory
//   warp 4     the weights (TMA) and a stage's count of bytes
//   warp 5     the MMAs (A stored [R][K] is K-major; B stored [N][R] has R
//              contiguous, an MN-major operand: no transposed copy)
// ---------------------------------------------------------------------------
constexpr int SHR_THREADS = 192;
constexpr int SHR_MOST = 6;  // stages at most

// One stage's weights: Rp rows of A, or 64 rows of B in 64-column boxes; as many stages as leave room for two CTAs
// on an SM (one for ranks above 64).
__host__ __device__ inline int shrink_wbytes(int R, bool grads) {
  return R > 64 ? 2 * HALF : (grads ? HALF : ((R + 15) & ~15) * 128);
}
__host__ __device__ inline int shrink_stages(int R, bool grads) {
  const int n = (R > 64 ? 220 * 1024 : 111 * 1024) / (BOX + shrink_wbytes(R, grads));
  return n < SHR_MOST ? n : SHR_MOST;
}
__host__ __device__ inline size_t shrink_smem(int R, bool grads) {
  return 1024 + (size_t)shrink_stages(R, grads) * (BOX + shrink_wbytes(R, grads));
}
__host__ __device__ inline uint32_t tmem_cols(int c) { return c <= 32 ? 32 : c <= 64 ? 64 : c <= 128 ? 128 : 256; }

__global__ void __launch_bounds__(SHR_THREADS, 2) k_lora_shrink(const Args a, const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t dsmem[];
  __shared__ uint64_t full[SHR_MOST], empty[SHR_MOST], acc_full;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_addr(dsmem) + 1023u) & ~1023u;
  uint8_t* const basep = dsmem + (base - smem_addr(dsmem));
  volatile int* abort = &abort_flag;
  int* status = a.hdr + H_STATUS;
  const bool grads = gridDim.z > 1;
  const int ST = shrink_stages(a.R, grads), stage = BOX + shrink_wbytes(a.R, grads);
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 129);  // 128 threads' copies of token rows, the weights' expect-tx arrival
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();
  const int tile = blockIdx.y;
  const int2 tl = __ldcg(a.tiles + tile);
  // rows of this thread's copies: i * 4 + lane / 8 of its warp's 32
  int tok[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) tok[i] = __ldcg(a.rowmap + tile * TM + (warp & 3) * 32 + i * 4 + (lane >> 3));
  if (tl.x < 0) return;  // the whole cluster leaves: nothing waits for it (a tile past the last has no rows either)
  const bool grad = blockIdx.z != 0;
  const int S = gridDim.x, rank = blockIdx.x;
  const int D = grad ? a.N : a.K, KB = (D + BK - 1) / BK;
  const int kb0 = rank * KB / S, nkb = (rank + 1) * KB / S - kb0;
  const uint32_t cols = tmem_cols(a.Rp);
  if (warp == 5) tmem_alloc(&tmem_base, cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  float* part = reinterpret_cast<float*>(basep);
  const int PP = a.Rp + 4;  // row pitch of the partial sums, padded by 16 bytes
  if (warp < 4) {
    const uint16_t* src = grad ? a.dy : a.x;
    const int ld = grad ? a.lddy : a.ldx;
    const int c8 = (lane & 7) * 8;
    const bool any = warp * 32 < tl.y;
    // 32 neighbouring tokens (a group's tokens are in ascending order): one box of them
    const int tok0 = __shfl_sync(0xffffffffu, tok[0], 0);
    const bool box = warp * 32 + 32 <= tl.y && __shfl_sync(0xffffffffu, tok[7], 31) - tok0 == 31;
    const CUtensorMap* xm = grad ? &maps.dy32 : &maps.x32;
    uint32_t dst[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) dst[i] = base + sw128_off(warp * 32 + i * 4 + (lane >> 3), c8);
    for (int i = 0; i < nkb; ++i) {
      const int s = i % ST, col = (kb0 + i) * BK;
      const bool ok = i < ST || wait_ab(&empty[s], ((i / ST) - 1) & 1, abort, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (box) {
        if (lane == 0) {
          mbar_expect_tx(&full[s], 32 * 128);
          tma_load_2d(base + s * stage + warp * 32 * 128, xm, col, tok0, &full[s]);
        }
        mbar_arrive(&full[s]);
        continue;
      }
      if (any) {
        const bool in = col + c8 < D;
        const uint16_t* at = src + (in ? col + c8 : 0);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          cp_async16(dst[j & 1] + s * stage + (j >> 1) * 1024, at + (int64_t)tok[j] * ld, in ? 16u : 0u);
      }
      cp_async_arrive(&full[s]);
    }
    cp_async_wait<0>();
    // Every CTA's sums to its shared memory (the stages are free by then), [128][Rp].
    bool ok = wait_ab(&acc_full, 0, abort, status);
    ok = __all_sync(0xffffffffu, ok);
    if (ok && any) {
      tc_fence_after();
      const int r = warp * 32 + lane;
      for (int c = 0; c < a.Rp; c += 16) {
        uint32_t v[16];
        tc_ld16(tmem + ((uint32_t)(warp * 32) << 16) + (uint32_t)c, v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(part + r * PP + c + 4 * j) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
      tc_fence_before();
    }
  } else if (warp == 4) {
    const uint32_t tx = grad ? (a.R > 64 ? 2 : 1) * HALF : a.Rp * 128;
    int i = 0;
    if (lane == 0) {
      for (; i < nkb; ++i) {
        const int s = i % ST, col = (kb0 + i) * BK;
        if (i >= ST && !wait_ab(&empty[s], ((i / ST) - 1) & 1, abort, status)) break;
        const uint32_t wsm = base + s * stage + BOX;
        mbar_arrive_expect_tx(&full[s], tx);
        if (grad) {
          tma_load_3d(wsm, &maps.b, 0, col, tl.x, &full[s]);
          if (a.R > 64) tma_load_3d(wsm + HALF, &maps.b, 64, col, tl.x, &full[s]);
        } else {
          tma_load_3d(wsm, &maps.a, col, 0, tl.x, &full[s]);
        }
      }
      // the CTA's memory must outlive every copy in flight
      for (int r = (i > ST ? i - ST : 0); r < i; ++r) mbar_drain(&full[r % ST], (r / ST) & 1);
    }
  } else {
    const uint32_t idesc = idesc_f32acc(TM, a.Rp, true) | (grad ? IDESC_B_MN : 0u);
    int i = 0;
    for (; i < nkb; ++i) {
      const int s = i % ST;
      const bool ok = wait_ab(&full[s], (i / ST) & 1, abort, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_proxy_async();  // the copies that arrived -> visible to the tensor core
      tc_fence_after();
      if (elect_one()) {
        const uint32_t xs = base + s * stage, wsm = xs + BOX;
        const uint64_t ad = sw128_desc(xs);
        const uint64_t bd = grad ? sw128_desc_mn(wsm, HALF) : sw128_desc(wsm);
        const uint64_t bstep = grad ? 2048 >> 4 : 32 >> 4;  // 16 rows of B, or 16 columns of A
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc_mma(tmem, ad + (uint64_t)(ks * 2), bd + ks * bstep, idesc, (i > 0 || ks > 0) ? 1u : 0u);
        tc_commit(&empty[s]);
        if (i == nkb - 1) tc_commit(&acc_full);
      }
      __syncwarp();
    }
    for (int r = (i > ST ? i - ST : 0); r < i; ++r) mbar_drain(&empty[r % ST], (r / ST) & 1);
  }
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_free(tmem, cols);
  }
  // The CTAs' sums of this CTA's share of the rows, all asked for at once and added in CTA order.
  if (S > 1) cluster_sync();
  const int rows = TM / S, r0 = rank * rows, R4 = a.R / 4;
  const float sc = __ldg(a.scale + tl.x);
  uint16_t* hi = grad ? a.g : a.h;
  uint16_t* lo = hi + (size_t)a.max_tiles * TM * a.R;
  const uint32_t part_s = base;
  auto reduce = [&](auto s_) {  // for a cluster of that many CTAs: eight loads in flight
    constexpr int SS = decltype(s_)::value, U = 8 / SS;
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < rows * R4; i0 += SHR_THREADS * U) {
      float4 u[U][SS];
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int i = i0 + e * SHR_THREADS, r = r0 + i / R4, c = (i % R4) * 4;
#pragma unroll
        for (int q = 0; q < SS; ++q) {
          u[e][q] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i < rows * R4 && r < tl.y) u[e][q] = ld_dsmem_f4(dsmem_addr(part_s + (uint32_t)(r * PP + c) * 4, q));
        }
      }
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int i = i0 + e * SHR_THREADS, r = r0 + i / R4, c = (i % R4) * 4;
        if (i >= rows * R4) break;
        float4 v = u[e][0];
#pragma unroll
        for (int q = 1; q < SS; ++q) {
          v.x += u[e][q].x;
          v.y += u[e][q].y;
          v.z += u[e][q].z;
          v.w += u[e][q].w;
        }
        v.x *= sc;
        v.y *= sc;
        v.z *= sc;
        v.w *= sc;
        uint2 hv, lv;
        halves(v, hv, lv);
        const size_t at = ((size_t)tile * TM + r) * a.R + c;
        *reinterpret_cast<uint2*>(hi + at) = hv;
        *reinterpret_cast<uint2*>(lo + at) = lv;
      }
    }
  };
  if (S == 8)
    reduce(std::integral_constant<int, 8>());
  else if (S == 4)
    reduce(std::integral_constant<int, 4>());
  else if (S == 2)
    reduce(std::integral_constant<int, 2>());
  else
    reduce(std::integral_constant<int, 1>());
  if (S > 1) cluster_sync();  // the others' shared memory stays until it has been read
}

// ---------------------------------------------------------------------------
// Expand: out = bf16(in + h B^T) (GRAD: in + g A), per tile [128 x R] times
// [R x 128 columns] for both halves of h. The (tile, 128 columns) items are one
// list, and each CTA takes a run of it, so that a tile's h is loaded once per run.
// Bound by the base rows it reads and the rows it writes: those go through each
// epilogue warp's own ring of shared memory (32 rows x 32 columns an item, up
// to three items ahead), without any barrier. Sixteen epilogue warps: with eight
// of twice the width an item took 3500 cycles at 42 % of the issue slots. 46.7 us
// alone for 8192 tokens, 8192 columns, rank 64 (268 MB: 5.7 TB/s, 0.85 of a copy).
//   warp 0      weights and a tile's h (TMA)
//   warp 1      the MMAs into two accumulators of 128 columns
//   warps 2-17  base rows (asynchronous copies); tensor memory + base -> bf16 in
//               place in shared memory -> 64-byte pieces of rows
// ---------------------------------------------------------------------------
constexpr int EXP_WARPS = 16;  // epilogue warps
constexpr int EXP_THREADS = 64 + 32 * EXP_WARPS;
constexpr int YSLOT = 32 * 64;  // one warp's rows of an item
// Byte offset of 16-byte piece c of row r of a warp's rows: two rows to 128 bytes, pieces swizzled by row pair, so
// that eight rows' same pieces, and two rows' all pieces, each touch every bank once.
__device__ __forceinline__ uint32_t yoff(int r, int c) { return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)); }
__host__ __device__ inline int exp_hbufs(int R) { return R > 64 ? 1 : 2; }
__host__ __device__ inline int exp_yslots(int R) { return R > 64 ? 3 : 4; }
__host__ __device__ inline int exp_wbytes(int R) { return R > 64 ? 2 * BOX : BOX; }      // one stage's weights
__host__ __device__ inline int exp_hbytes(int R) { return R > 64 ? 4 * BOX : 2 * BOX; }  // hi and lo of a tile
__host__ __device__ inline size_t exp_smem(int R) {
  return 1024 + (size_t)2 * exp_wbytes(R) + (size_t)exp_hbufs(R) * exp_hbytes(R) + (size_t)exp_yslots(R) * EXP_WARPS * YSLOT;
}

template <bool GRAD, bool WIDE>  // WIDE: rank above 64
__global__ void __launch_bounds__(EXP_THREADS, 1) k_lora_expand(const Args a, const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t dsmem[];
  __shared__ uint64_t full[2], empty[2], acc_full[2], acc_empty[2], h_full[2], h_empty[2];
  __shared__ uint64_t y_full[EXP_WARPS][4];  // a warp's slots filled by TMA
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  constexpr int ANY_R = WIDE ? 128 : 64;
  constexpr int HB = WIDE ? 1 : 2, nbox = WIDE ? 2 : 1, YS = WIDE ? 3 : 4, LY = YS - 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_addr(dsmem) + 1023u) & ~1023u;
  uint8_t* const basep = dsmem + (base - smem_addr(dsmem));
  volatile int* abort = &abort_flag;
  int* status = a.hdr + H_STATUS;
  const int stage = exp_wbytes(ANY_R), hbytes = exp_hbytes(ANY_R);
  const uint32_t hbase = base + 2 * stage, ybase = hbase + HB * hbytes;
  const int D = GRAD ? a.K : a.N, nsub = (D + 127) / 128;
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&full[b], 1);
      mbar_init(&empty[b], 1);
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], EXP_WARPS);
      mbar_init(&h_full[b], 1);
      mbar_init(&h_empty[b], 1);
    }
    for (int w = 0; w < EXP_WARPS; ++w)
      for (int i = 0; i < YS; ++i) mbar_init(&y_full[w][i], 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  pdl_trigger();
  // The plan is complete (the kernel before lets this one start only after its own wait), and so are the base rows;
  // only h has to be waited for, by the warp that loads it.
  // This CTA's run [u0, u1) of the items: tile u / nsub, columns 128 (u % nsub) ...
  const long long items = (long long)__ldcg(a.hdr + H_TILES) * nsub;
  const int u0 = (int)(items * blockIdx.x / gridDim.x), u1 = (int)(items * (blockIdx.x + 1) / gridDim.x);
  const int tile0 = u0 / nsub, sub0 = u0 - tile0 * nsub;
  const size_t plane = (size_t)a.max_tiles * TM;
  if (warp == 0) {
    if (lane == 0) {
      pdl_wait();
      int m = 0, hn = 0;  // items with an adapter, h loads
      int tile = tile0, sub = sub0;
      int2 tl = make_int2(-1, 0);
      for (int u = u0; u < u1; ++u, ++sub) {
        if (sub == nsub) {
          sub = 0;
          ++tile;
        }
        const int col = sub * 128;
        if (u == u0 || sub == 0) {
          tl = __ldcg(a.tiles + tile);
          if (tl.x >= 0) {
            const int b = hn % HB;
            if (hn >= HB && !wait_ab(&h_empty[b], ((hn / HB) - 1) & 1, abort, status)) break;
            const CUtensorMap* mp = GRAD ? &maps.g : &maps.h;
            mbar_arrive_expect_tx(&h_full[b], (uint32_t)hbytes);
            for (int p = 0; p < 2; ++p)
              for (int x = 0; x < nbox; ++x)
                for (int y = 0; y < 2; ++y)
                  tma_load_2d(hbase + b * hbytes + (p * nbox + x) * BOX + y * HALF, mp, x * 64,
                              (int)(p * plane) + tile * TM + y * 64, &h_full[b]);
            ++hn;
          }
        }
        if (tl.x < 0) continue;
        const int s = m & 1;
        if (m >= 2 && !wait_ab(&empty[s], ((m >> 1) - 1) & 1, abort, status)) break;
        const uint32_t wsm = base + s * stage;
        const int boxes = col + 64 < D ? 2 : 1;  // 64-column halves that hold columns at all
        if (GRAD) {
          mbar_arrive_expect_tx(&full[s], (uint32_t)(boxes * a.Rp * 128));
          for (int y = 0; y < boxes; ++y) tma_load_3d(wsm + y * a.Rp * 128, &maps.a, col + 64 * y, 0, tl.x, &full[s]);
        } else {
          mbar_arrive_expect_tx(&full[s], (uint32_t)(boxes * nbox * HALF));
          for (int x = 0; x < nbox; ++x)
            for (int y = 0; y < boxes; ++y)
              tma_load_3d(wsm + x * BOX + y * HALF, &maps.b, x * 64, col + 64 * y, tl.x, &full[s]);
        }
        ++m;
      }
      for (int r = (m > 2 ? m - 2 : 0); r < m; ++r) mbar_drain(&full[r & 1], (r >> 1) & 1);
      for (int r = (hn > HB ? hn - HB : 0); r < hn; ++r) mbar_drain(&h_full[r % HB], (r / HB) & 1);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f32acc(TM, 128, true) | (GRAD ? IDESC_B_MN : 0u);
    int m = 0, hn = 0, tile = tile0, sub = sub0;
    int2 tl = make_int2(-1, 0);
    for (int u = u0; u < u1; ++u, ++sub) {
      bool ok = true;
      if (sub == nsub) {
        sub = 0;
        ++tile;
      }
      if (u == u0 || sub == 0) {
        tl = __ldcg(a.tiles + tile);
        if (tl.x >= 0) {
          ok = wait_ab(&h_full[hn % HB], (hn / HB) & 1, abort, status);
          ++hn;
        }
      }
      if (tl.x < 0) continue;
      const int b = m & 1, hb = (hn - 1) % HB;
      ok = ok && (m < 2 || wait_ab(&acc_empty[b], ((m >> 1) - 1) & 1, abort, status));
      ok = ok && wait_ab(&full[b], (m >> 1) & 1, abort, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t wsm = base + b * stage, hs = hbase + hb * hbytes, acc = tmem + b * 128;
        uint32_t on = 0;
        for (int p = 0; p < 2; ++p)
          for (int ks = 0; ks < a.Rp / 16; ++ks) {
            const uint64_t ad = sw128_desc(hs + (p * nbox + (ks >> 2)) * BOX) + (uint64_t)((ks & 3) * 2);
            const uint64_t bd = GRAD ? sw128_desc_mn(wsm + ks * 2048, a.Rp * 128)
                                     : sw128_desc(wsm + (ks >> 2) * BOX) + (uint64_t)((ks & 3) * 2);
            tc_mma(acc, ad, bd, idesc, on);
            on = 1;
          }
        tc_commit(&empty[b]);
        tc_commit(&acc_full[b]);
        if (u + 1 == u1 || sub + 1 == nsub) tc_commit(&h_empty[hb]);
      }
      __syncwarp();
      ++m;
    }
    for (int r = (m > 2 ? m - 2 : 0); r < m; ++r) mbar_drain(&acc_full[r & 1], (r >> 1) & 1);
  } else {
    const int q = warp & 3, c0 = ((warp - 2) >> 2) * 32;  // tensor-memory lanes 32 q .., columns c0 .. of an item
    const int rsub = lane >> 2, c8 = (lane & 3) * 8;      // this lane's place in a copy of eight rows
    const uint32_t ys = ybase + (uint32_t)((warp - 2) * YS * YSLOT);
    uint8_t* const yp = basep + (ys - base);
    uint64_t* const ybar = y_full[warp - 2];
    // Copies run LY items ahead: item (ptile, psub) goes to slot `pslot`, this warp's rows being tokens `p`. Two slots
    // more than that, so that a slot's last output rows have left it when it is filled again.
    int ptile = tile0, psub = sub0, pslot = 0, left = a.in ? u1 - u0 : 0;
    struct Rows {
      int tok[4];  // tokens of rows i * 8 + rsub
      int first;   // all 32 rows are the tokens from here on, or -1
      int count;   // rows of the warp that are the tile's
    };
    auto rows_of = [&](int tile, Rows& r) {
      const int count = __ldcg(&a.tiles[tile].y);
#pragma unroll
      for (int i = 0; i < 4; ++i) r.tok[i] = __ldcg(a.rowmap + tile * TM + q * 32 + i * 8 + rsub);
      const int lo = __shfl_sync(0xffffffffu, r.tok[0], 0), hi = __shfl_sync(0xffffffffu, r.tok[3], 31);
      r.count = count - q * 32;
      r.first = r.count >= 32 && hi - lo == 31 ? lo : -1;  // (a group's tokens are in ascending order)
    };
    Rows p = {};
    if (left > 0) rows_of(ptile, p);
    const uint32_t off = yoff(rsub, lane & 3);  // this lane's place in eight rows (512 bytes)
    uint32_t phase = 0;                         // bit s: parity of slot s's next fill by TMA
    auto fetch = [&]() {
      if (left > 0) {
        if (psub == nsub) {
          psub = 0;
          ++ptile;
          rows_of(ptile, p);
        }
        const int col = psub * 128 + c0;
        if (p.count > 0 && col < D) {
          const uint32_t slot = ys + (uint32_t)pslot * YSLOT;
          if (p.first >= 0) {
            if (lane == 0) {
              mbar_arrive_expect_tx(&ybar[pslot], YSLOT);
              tma_load_2d(slot, &maps.in, col, p.first, &ybar[pslot]);
            }
          } else {
            const bool in = col + c8 < D;
            const uint16_t* src = a.in + (in ? col + c8 : 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async16(slot + off + i * 512, src + (int64_t)p.tok[i] * a.ldo, in ? 16u : 0u);
          }
        }
        ++psub;
        --left;
        pslot = pslot + 1 == YS ? 0 : pslot + 1;
      }
      cp_async_commit();
    };
    int m = 0, tile = tile0, sub = sub0, slot_i = 0;
    Rows r = {};
    int2 tl = make_int2(-1, 0);
#pragma unroll
    for (int i = 0; i < LY; ++i) fetch();
    for (int u = u0; u < u1; ++u, ++sub) {
      if (sub == nsub) {
        sub = 0;
        ++tile;
      }
      if (u == u0 || sub == 0) {
        tl = __ldcg(a.tiles + tile);
        rows_of(tile, r);
      }
      const int col = sub * 128 + c0;
      const bool mma = tl.x >= 0, live = r.count > 0 && col < D;  // live: this warp's rows and columns hold something
      const int b = m & 1;
      uint32_t w[32];
      bool ok = true;
      if (mma) {
        ok = wait_ab(&acc_full[b], (m >> 1) & 1, abort, status);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        if (live) {
          tc_ld32_async(tmem + b * 128 + c0 + ((uint32_t)(q * 32) << 16), w);
          tc_wait_ld();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&acc_empty[b]);  // the accumulator is free for the MMAs
          bulk_wait_read<1>();         // the output of two items ago has left the slot that is filled next
        }
        ++m;
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j] = 0u;
        if (lane == 0) bulk_wait_read<1>();
      }
      __syncwarp();
      fetch();
      if (live && a.in && r.first >= 0) {
        ok = wait_ab(&ybar[slot_i], (phase >> slot_i) & 1, abort, status);
        phase ^= 1u << slot_i;
        if (!__all_sync(0xffffffffu, ok)) break;
      }
      cp_async_wait<LY>();
      __syncwarp();
      if (live) {
        uint8_t* slot = yp + slot_i * YSLOT;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4* at = reinterpret_cast<uint4*>(slot + yoff(lane, j));
          uint4 y = make_uint4(0u, 0u, 0u, 0u);
          if (a.in) y = *at;
          const uint32_t* d = &w[8 * j];
          y.x = f2b2(bf16lo(y.x) + __uint_as_float(d[0]), bf16hi(y.x) + __uint_as_float(d[1]));
          y.y = f2b2(bf16lo(y.y) + __uint_as_float(d[2]), bf16hi(y.y) + __uint_as_float(d[3]));
          y.z = f2b2(bf16lo(y.z) + __uint_as_float(d[4]), bf16hi(y.z) + __uint_as_float(d[5]));
          y.w = f2b2(bf16lo(y.w) + __uint_as_float(d[6]), bf16hi(y.w) + __uint_as_float(d[7]));
          *at = y;
        }
        if (r.first >= 0) {
          fence_proxy_async();  // these stores -> visible to TMA
          __syncwarp();
          if (lane == 0) tma_store_2d(&maps.out, col, r.first, ys + slot_i * YSLOT);
        } else {
          __syncwarp();
          if (col + c8 < D) {
            uint16_t* dst = a.out + col + c8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 y = lds128(slot + off + i * 512);
              if (i * 8 + rsub < r.count) *reinterpret_cast<uint4*>(dst + (int64_t)r.tok[i] * a.ldo) = y;
            }
          }
          fence_proxy_async();  // these accesses come before a box that may fill the slot next
        }
      }
      if (lane == 0) bulk_commit();
      slot_i = slot_i + 1 == YS ? 0 : slot_i + 1;
    }
    cp_async_wait<0>();
    if (lane == 0) bulk_wait_all();
    // after a failed wait, boxes may still be on their way into this warp's slots
    if (*abort && lane == 0)
      for (int i = 0; i < YS; ++i) mbar_drain(&ybar[i], (phase >> i) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 256);
  }
}

// ---------------------------------------------------------------------------
// Weights' gradients: for a chunk of one adapter's tiles and a 128-wide slab of K
// (dA) or of N (dB), [slab x tokens] times [tokens x R] on the tensor cores. Both
// operands lie with the reduction (the tokens) as rows, so both are MN-major and
// x, dy, g, h are used as they lie in memory. A chunk that is its adapter's only
// one writes bf16 itself; the others leave FP32 partial sums, which k_lora_dw_sum
// adds in chunk order. Bound by the rows of x and dy, of which L2 still holds those
// that the shrink read last: 20.4 us alone and cold for 8192 tokens of 2048 x 2048,
// rank 32 (67 MB: 3.3 TB/s), and 5.6 us for the sums.
//   warps 0-3 token rows, then the accumulator (a thread is one column of the
//   slab); warp 4 g or h (TMA); warp 5 the MMAs
// ---------------------------------------------------------------------------
constexpr int DW_THREADS = 192;
__host__ __device__ inline int dw_stages(int R) { return R > 64 ? 2 : 3; }
__host__ __device__ inline int dw_stage_bytes(int R) { return 2 * HALF + (R > 64 ? 4 : 2) * HALF; }
__host__ __device__ inline size_t dw_smem(int R) { return 1024 + (size_t)dw_stages(R) * dw_stage_bytes(R); }

template <bool WIDE>
__global__ void __launch_bounds__(DW_THREADS, 2) k_lora_dw(const Args a, const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t dsmem[];
  __shared__ uint64_t full[3], empty[3], acc_full;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  constexpr int ST = WIDE ? 2 : 3, nbox = WIDE ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_addr(dsmem) + 1023u) & ~1023u;
  volatile int* abort = &abort_flag;
  int* status = a.hdr + H_STATUS;
  const int stage = dw_stage_bytes(WIDE ? 128 : 64);
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 129);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();
  const int slab = blockIdx.x;
  if ((int)blockIdx.y >= __ldcg(a.hdr + H_CHUNKS)) return;
  const int4 ch = __ldcg(a.chunks + blockIdx.y);
  const bool is_b = slab >= a.slabs_a;
  const int D = is_b ? a.N : a.K, col0 = (is_b ? slab - a.slabs_a : slab) * 128;
  const int last = __ldcg(a.tiles + ch.y + ch.z - 1).y;
  const int steps = 2 * (ch.z - 1) + (last > 64 ? 2 : 1);  // half tiles of 64 tokens
  const int rows = TM * (ch.z - 1) + last;
  const uint32_t cols = tmem_cols(a.Rp);
  if (warp == 5) tmem_alloc(&tmem_base, cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  if (warp < 4) {
    // Rows 16 warp .. + 15 of a half tile, two rows of 256 bytes a copy: lane = row parity, 16-byte piece.
    const uint16_t* src = is_b ? a.dy : a.x;
    const int ld = is_b ? a.lddy : a.ldx;
    const int c8 = (lane & 15) * 8;
    const bool in = col0 + c8 < D;
    src += in ? col0 + c8 : 0;
    const int* map = a.rowmap + ch.y * TM + warp * 16 + (lane & 15);
    const CUtensorMap* xm = is_b ? &maps.dy16 : &maps.x16;
    const int boxes = col0 + 64 < D ? 2 : 1;  // 64-column halves that hold columns at all
    int tok = __ldcg(map);
    for (int i = 0; i < steps; ++i) {
      const int s = i % ST;
      const int next = i + 1 < steps ? __ldcg(map + (i + 1) * 64) : 0;
      const bool ok = i < ST || wait_ab(&empty[s], ((i / ST) - 1) & 1, abort, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint32_t xs = base + s * stage;
      const int tok0 = __shfl_sync(0xffffffffu, tok, 0);
      // 16 neighbouring tokens (ascending, none of them a repeat): boxes of them
      if (i * 64 + warp * 16 + 16 <= rows && __shfl_sync(0xffffffffu, tok, 15) - tok0 == 15) {
        if (lane == 0) {
          mbar_expect_tx(&full[s], boxes * 16 * 128);
          for (int y = 0; y < boxes; ++y) tma_load_2d(xs + y * HALF + warp * 16 * 128, xm, col0 + 64 * y, tok0, &full[s]);
        }
        mbar_arrive(&full[s]);
        tok = next;
        continue;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = 2 * j + (lane >> 4);
        const int t = __shfl_sync(0xffffffffu, tok, r);
        cp_async16(xs + (lane & 8 ? HALF : 0) + sw128_off(warp * 16 + r, c8 & 63), src + (int64_t)t * ld, in ? 16u : 0u);
      }
      cp_async_arrive(&full[s]);
      tok = next;
    }
    cp_async_wait<0>();
    bool ok = wait_ab(&acc_full, 0, abort, status);
    ok = __all_sync(0xffffffffu, ok);
    const int col = col0 + warp * 32 + lane;
    if (ok && col0 + warp * 32 < D) {
      tc_fence_after();
      float* part = ch.w >= 0 ? a.part + (size_t)ch.w * a.R * (a.K + a.N) + (is_b ? (size_t)a.R * a.K : 0) : nullptr;
      uint16_t* out = is_b ? a.dB + (size_t)ch.x * a.N * a.R : a.dA + (size_t)ch.x * a.R * a.K;
      for (int c = 0; c < a.Rp; c += 16) {
        uint32_t v[16];
        tc_ld16(tmem + ((uint32_t)(warp * 32) << 16) + (uint32_t)c, v);
        if (col >= D) continue;
        if (is_b) {  // [N][R]: a thread's row
#pragma unroll
          for (int j = 0; j < 16; j += 8) {
            if (c + j >= a.R) break;
            const size_t at = (size_t)col * a.R + c + j;
            if (part) {
              *reinterpret_cast<uint4*>(part + at) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
              *reinterpret_cast<uint4*>(part + at + 4) = make_uint4(v[j + 4], v[j + 5], v[j + 6], v[j + 7]);
            } else {
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] = f2b2(__uint_as_float(v[j + 2 * e]), __uint_as_float(v[j + 2 * e + 1]));
              *reinterpret_cast<uint4*>(out + at) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        } else {  // [R][K]: a warp's 32 neighbours of each rank row
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (c + j >= a.R) break;
            const size_t at = (size_t)(c + j) * a.K + col;
            if (part)
              part[at] = __uint_as_float(v[j]);
            else
              out[at] = f2b(__uint_as_float(v[j]));
          }
        }
      }
      tc_fence_before();
    }
  } else if (warp == 4) {
    if (lane == 0) {
      const size_t plane = (size_t)a.max_tiles * TM;
      const CUtensorMap* gm = is_b ? &maps.h : &maps.g;
      int i = 0;
      for (; i < steps; ++i) {
        const int s = i % ST, row0 = ch.y * TM + i * 64;
        if (i >= ST && !wait_ab(&empty[s], ((i / ST) - 1) & 1, abort, status)) break;
        const uint32_t gs = base + s * stage + 2 * HALF;
        mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * nbox * HALF));
        for (int p = 0; p < 2; ++p)
          for (int x = 0; x < nbox; ++x)
            tma_load_2d(gs + (p * nbox + x) * HALF, gm, x * 64, (int)(p * plane) + row0, &full[s]);
      }
      for (int r = (i > ST ? i - ST : 0); r < i; ++r) mbar_drain(&full[r % ST], (r / ST) & 1);
    }
  } else {
    const uint32_t idesc = idesc_f32acc(TM, a.Rp, true) | IDESC_A_MN | IDESC_B_MN;
    int i = 0;
    for (; i < steps; ++i) {
      const int s = i % ST;
      const bool ok = wait_ab(&full[s], (i / ST) & 1, abort, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_proxy_async();  // the copies that arrived -> visible to the tensor core
      tc_fence_after();
      if (elect_one()) {
        const uint32_t xs = base + s * stage, gs = xs + 2 * HALF;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc_mma(tmem, sw128_desc_mn(xs + ks * 2048, HALF), sw128_desc_mn(gs + p * nbox * HALF + ks * 2048, HALF), idesc,
                   (i > 0 || p > 0 || ks > 0) ? 1u : 0u);
        tc_commit(&empty[s]);
        if (i == steps - 1) tc_commit(&acc_full);
      }
      __syncwarp();
    }
    for (int r = (i > ST ? i - ST : 0); r < i; ++r) mbar_drain(&empty[r % ST], (r / ST) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_free(tmem, cols);
  }
}

// Gradients of the adapters with several chunks (their partial sums, in chunk order) or none (zero).
__global__ void __launch_bounds__(256) k_lora_dw_sum(const Args a) {
  pdl_wait();
  const int2 of = __ldcg(a.of_adapter + blockIdx.y);
  if (of.y == 1) return;
  const size_t na = (size_t)a.R * a.K, all = na + (size_t)a.N * a.R;
  const float* p = a.part + (size_t)of.x * all;
  uint16_t* dA = a.dA + blockIdx.y * na;
  uint16_t* dB = a.dB + blockIdx.y * (all - na);
  for (size_t e = 8 * ((size_t)blockIdx.x * 256 + threadIdx.x); e < all; e += (size_t)gridDim.x * 2048) {
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < of.y; ++c) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(p + c * all + e));
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p + c * all + e) + 1);
      s[0] += u.x, s[1] += u.y, s[2] += u.z, s[3] += u.w;
      s[4] += v.x, s[5] += v.y, s[6] += v.z, s[7] += v.w;
    }
    const uint4 o = make_uint4(f2b2(s[0], s[1]), f2b2(s[2], s[3]), f2b2(s[4], s[5]), f2b2(s[6], s[7]));
    *reinterpret_cast<uint4*>(e < na ? dA + e : dB + (e - na)) = o;  // R K is a multiple of 8: no piece straddles
  }
}

// ---------------------------------------------------------------------------
// Up to 32 rows (decode). One cluster of FEW_S CTAs for each distinct adapter of
// the call: CTA s takes a run of the 32-column steps of K for h = A x, the CTAs'
// sums meet in distributed shared memory (added in CTA order), and each takes its
// share of the N rows of B for B h. With so few rows every weight is used once,
// so weights go from memory to tensor-core fragments in registers, 16 (or 8)
// bytes a lane; mma.sync with the weights as its 16 rows and the tokens as its 8
// columns. The order of the columns within a step is the same for both operands
// of a product and otherwise free, so a lane's neighbouring columns need no
// shuffling. A CTA's share of B is one run of memory: it comes into shared memory
// in pieces of 256 rows with bulk copies that start before A is read (from L2 into
// registers it took 10 of 21 us for 32 adapters of rank 64, 2048 x 8192). Bound by
// latency for one adapter (6.4 us alone and cold: 2048 x 2048, rank 16), by the adapters' bytes for
// many (15.0 us alone and cold for those 32: 42 MB, 2.8 TB/s).
// ---------------------------------------------------------------------------
constexpr int FEW = MAX_BATCH;
constexpr int FEW_S = 8;
constexpr int FEW_THREADS = 256;

struct FewArgs {
  int K, N, R, n, T;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  const int* adapter;
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* in;  // base rows (bf16) or null
  uint16_t* out;       // bf16 rows, or
  float* out32;        // FP32 rows [T][N] of B h alone
  int64_t ldo;
  int with_none;  // rows without an adapter are copied too
  int* status;
  int clear;      // the status word starts at zero
  size_t smem;    // of the launch
};

__host__ __device__ inline int few_rt(int R) { return (R + 15) / 16; }  // 16-row tiles of the rank
// Warps side by side over the rank's tiles; the rest of the eight split the columns.
__host__ __device__ inline int few_wr(int R) { return few_rt(R) >= 8 ? 8 : few_rt(R) >= 4 ? 4 : few_rt(R) >= 2 ? 2 : 1; }
// Shared memory: pieces of B, the column splits' sums [8 / wr][tokens][rank], the CTA's sums [tokens][rank], h as two
// bf16 halves. Together a third of an SM's where two pieces leave that.
constexpr int FEW_PIECE = 256;  // rows of a piece: two tiles of 16 for each warp
constexpr int FEW_MOST = 8;     // pieces at once
constexpr int FEW_CTAS = 3;     // CTAs of an SM at most (shared memory holds two of rank 64 with 16 rows, one of rank 128)
constexpr size_t FEW_SMEM = 224 * 1024 / FEW_CTAS;
__host__ __device__ inline int few_pieces(int N) { return ((N + 15) / 16 + FEW_S * 16 - 1) / (FEW_S * 16); }  // of a CTA's share, at most
struct FewPlan {
  int RP;      // rank padded to 16
  int pieces;  // held at once
  size_t red, part, hs, total;
};
// `cols`: tokens it is laid out for; `most`: pieces of a CTA's share; `budget`: bytes.
__host__ __device__ inline FewPlan few_plan(int R, int cols, int most, size_t budget) {
  FewPlan p;
  p.RP = few_rt(R) * 16;
  const size_t rest = sizeof(float) * (8 / few_wr(R) + 1) * cols * p.RP + (size_t)2 * 2 * cols * (p.RP + 8);
  const size_t piece = (size_t)FEW_PIECE * R * 2;
  const int fit = rest + 2 * piece > budget ? 2 : (int)((budget - rest) / piece);
  const int cap = most < FEW_MOST ? most : FEW_MOST;
  p.pieces = fit > cap ? cap : fit;
  size_t o = p.pieces * piece;
  p.red = o;   o += sizeof(float) * (8 / few_wr(R)) * cols * p.RP;
  p.part = o;  o += sizeof(float) * cols * p.RP;
  p.hs = o;    o += (size_t)2 * 2 * cols * (p.RP + 8);
  p.total = o;
  return p;
}

// What the two products of a group share.
struct FewGroup {
  const uint16_t* A;  // the adapter's
  const uint16_t* B;
  int count;           // tokens
  int n0, n1;          // this CTA's 16-row tiles of B
  int k0, k1;          // and its 32-column steps of K
  int cols;            // tokens that the shared memory is laid out for
};

// h = A x over this CTA's columns, this warp's share of it, into red[split][token][rank]. NT: token tiles of 8.
template <int NT>
__device__ __forceinline__ void few_shrink(const FewArgs& a, const FewGroup& G, const int* toks, float* red, int RP, int warp,
                                           int lane) {
  const int g = lane >> 2, t4 = lane & 3;
  const int wr = few_wr(a.R), wk = 8 / wr, wri = warp % wr, wki = warp / wr, RT = few_rt(a.R);
  const uint16_t* xr[NT];  // row of token 8 nt + g (past the count: the last token's)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) xr[nt] = a.x + toks[min(nt * 8 + g, G.count - 1)] * a.ldx + t4 * 8;
  for (int rt = wri; rt < RT; rt += wr) {
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
    const int r0 = rt * 16 + g, r1 = r0 + 8;
    const uint16_t* p0 = G.A + (int64_t)r0 * a.K + t4 * 8;
    const uint16_t* p1 = G.A + (int64_t)r1 * a.K + t4 * 8;
#pragma unroll 4
    for (int k = G.k0 + wki; k < G.k1; k += wk) {
      const int c = k * 32;
      const bool in = c + t4 * 8 < a.K;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      const uint4 u = in && r0 < a.R ? __ldg(reinterpret_cast<const uint4*>(p0 + c)) : zero;
      const uint4 v = in && r1 < a.R ? __ldg(reinterpret_cast<const uint4*>(p1 + c)) : zero;
      const uint32_t f0[4] = {u.x, v.x, u.y, v.y}, f1[4] = {u.z, v.z, u.w, v.w};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 xv = in ? ld_cg_v4(xr[nt] + c) : zero;
        mma_bf16(acc[nt], f0, xv.x, xv.y);
        mma_bf16(acc[nt], f1, xv.z, xv.w);
      }
    }
    const bool upper = rt * 16 + 8 < a.R;  // places past the rank are zero also beside an infinite x
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float* o = red + ((size_t)wki * G.cols + nt * 8 + 2 * t4) * RP + rt * 16 + g;
      o[0] = acc[nt][0];
      o[RP] = acc[nt][1];
      o[8] = upper ? acc[nt][2] : 0.f;
      o[RP + 8] = upper ? acc[nt][3] : 0.f;
    }
  }
}

// B h for this CTA's rows, piece by piece: warp w takes the 16-row tiles w and w + 8 of a piece at once, STEP columns of
// the rank a step. fetch(i) asks for piece i (thread 0).
template <int NT, int STEP, typename Fetch>
__device__ __forceinline__ void few_expand(const FewArgs& a, const FewGroup& G, const int* toks, const uint8_t* smem,
                                           const uint16_t* hs, const FewPlan& P, uint64_t* full, uint64_t* empty, int npieces,
                                           int warp, int lane, Fetch fetch) {
  const int g = lane >> 2, t4 = lane & 3;
  constexpr int LC = STEP / 4;  // neighbouring columns of a lane
  constexpr int ACC = NT == 1 ? 2 : 1;  // chains of MMAs: the halves of h apart, where registers allow
  const int HP = P.RP + 8;
  const uint16_t* lo = hs + G.cols * HP;
  const int end = min(G.n1 * 16, a.N);
  // lane: rows g, g + 8 of tokens 8 nt + 2 t4, + 1
  int64_t at[NT][2];  // first elements of those tokens' output rows, -1: none
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = nt * 8 + 2 * t4 + e;
      at[nt][e] = j < G.count ? toks[j] * (a.out32 ? (int64_t)a.N : a.ldo) : -1;
    }
  for (int i = 0; i < npieces; ++i) {
    const int sl = i % P.pieces, par = (i / P.pieces) & 1;
    // after a failed wait the piece is let land and used as it is: the status word tells
    if (!mbar_wait(&full[sl], par, a.status)) mbar_drain(&full[sl], par);
    const int row = G.n0 * 16 + i * FEW_PIECE + warp * 16 + g;
    bool in[4];  // rows row, + 8, + 128, + 136
#pragma unroll
    for (int q = 0; q < 4; ++q) in[q] = row + (q & 1) * 8 + (q >> 1) * 128 < end;
    const uint8_t* p = smem + (size_t)sl * FEW_PIECE * a.R * 2 + (size_t)((warp * 16 + g) * a.R + t4 * LC) * 2;
    float acc[2][ACC][NT][4];
#pragma unroll
    for (int z = 0; z < 2 * ACC * NT * 4; ++z) (&acc[0][0][0][0])[z] = 0.f;
#pragma unroll 2
    for (int c = 0; c < a.R; c += STEP) {
      uint4 w[4];  // STEP 16: two words of each
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        w[q] = make_uint4(0u, 0u, 0u, 0u);
        const uint8_t* pq = p + (size_t)((q & 1) * 8 + (q >> 1) * 128) * a.R * 2 + c * 2;
        if (STEP == 32) {
          if (in[q]) w[q] = lds128(pq);
        } else if (in[q] && c + t4 * LC < a.R) {
          const uint2 v = *reinterpret_cast<const uint2*>(pq);
          w[q].x = v.x, w[q].y = v.y;
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = (nt * 8 + g) * HP + c + t4 * LC;
        uint4 hv = make_uint4(0u, 0u, 0u, 0u), lv = hv;
        if (STEP == 32) {
          hv = *reinterpret_cast<const uint4*>(hs + h);
          lv = *reinterpret_cast<const uint4*>(lo + h);
        } else {
          const uint2 h2 = *reinterpret_cast<const uint2*>(hs + h), l2 = *reinterpret_cast<const uint2*>(lo + h);
          hv.x = h2.x, hv.y = h2.y, lv.x = l2.x, lv.y = l2.y;
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const uint32_t f0[4] = {w[2 * z].x, w[2 * z + 1].x, w[2 * z].y, w[2 * z + 1].y};
          const uint32_t f1[4] = {w[2 * z].z, w[2 * z + 1].z, w[2 * z].w, w[2 * z + 1].w};
          mma_bf16(acc[z][0][nt], f0, hv.x, hv.y);
          mma_bf16(acc[z][ACC - 1][nt], f0, lv.x, lv.y);
          if (STEP == 32) {
            mma_bf16(acc[z][0][nt], f1, hv.z, hv.w);
            mma_bf16(acc[z][ACC - 1][nt], f1, lv.z, lv.w);
          }
        }
      }
    }
    if (npieces > P.pieces) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[sl]);
      if (threadIdx.x == 0 && i + P.pieces < npieces) {
        mbar_wait(&empty[sl], par, a.status);
        fetch(i + P.pieces);
      }
    }
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (at[nt][e] < 0) continue;
          float v[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) v[q] = ACC == 2 ? acc[z][0][nt][e + 2 * q] + acc[z][ACC - 1][nt][e + 2 * q] : acc[z][0][nt][e + 2 * q];
          const int64_t o = at[nt][e] + row + z * 128;
          if (a.out32) {
            if (in[2 * z]) a.out32[o] = v[0];
            if (in[2 * z + 1]) a.out32[o + 8] = v[1];
          } else {
            if (in[2 * z]) a.out[o] = f2b((a.in ? __uint_as_float((uint32_t)a.in[o] << 16) : 0.f) + v[0]);
            if (in[2 * z + 1]) a.out[o + 8] = f2b((a.in ? __uint_as_float((uint32_t)a.in[o + 8] << 16) : 0.f) + v[1]);
          }
        }
  }
}

template <int NT, int STEP>  // tokens of a call: 8 NT at most; columns of the rank a step: 32 (multiples of it) or 16
__global__ void __launch_bounds__(FEW_THREADS, FEW_CTAS) k_lora_few(const FewArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int toks[FEW];
  __shared__ uint64_t full[FEW_MOST], empty[FEW_MOST];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < FEW_MOST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 8);
    }
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();
  if (a.clear && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.status = 0;
  // The blockIdx.y-th distinct adapter, by first use, and its tokens (every warp finds the same).
  int mine = lane < a.T ? __ldg(a.adapter + lane) : -2;
  if (mine < -1 || mine >= a.n) mine = lane < a.T ? -1 : -2;
  const unsigned same = __match_any_sync(0xffffffffu, mine);
  unsigned firsts = __ballot_sync(0xffffffffu, lane == __ffs(same) - 1 && mine != -2 && (mine >= 0 || a.with_none));
  for (int i = 0; i < (int)blockIdx.y; ++i) firsts &= firsts - 1;
  if (!firsts) return;  // fewer adapters than clusters: the whole cluster leaves
  const int lead = __ffs(firsts) - 1;
  const int ad = __shfl_sync(0xffffffffu, mine, lead);
  const unsigned set = __shfl_sync(0xffffffffu, same, lead);
  const int count = __popc(set);
  if (warp == 0 && ((set >> lane) & 1u)) toks[__popc(set & ((1u << lane) - 1))] = lane;
  __syncthreads();
  if (ad < 0) {  // no adapter: the base as it is
    for (int i = s * FEW_THREADS + threadIdx.x; i < count * (a.N / 8); i += FEW_S * FEW_THREADS) {
      const int t = toks[i / (a.N / 8)], c = i % (a.N / 8) * 8;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (a.in) v = *reinterpret_cast<const uint4*>(a.in + t * a.ldo + c);
      *reinterpret_cast<uint4*>(a.out + t * a.ldo + c) = v;
    }
    return;
  }
  // A group of up to 8 tokens needs less for its sums, and holds more of B.
  const int nt_used = (count + 7) >> 3, cols = nt_used == 1 ? 8 : 8 * NT;
  const FewPlan P = few_plan(a.R, cols, few_pieces(a.N), a.smem);
  float* red = reinterpret_cast<float*>(smem + P.red);
  float* part = reinterpret_cast<float*>(smem + P.part);
  uint16_t* hs = reinterpret_cast<uint16_t*>(smem + P.hs);
  const uint16_t* A = a.A + (int64_t)ad * a.R * a.K;
  const uint16_t* B = a.B + (int64_t)ad * a.N * a.R;
  const int ntiles = (a.N + 15) / 16, n0 = s * ntiles / FEW_S, n1 = (s + 1) * ntiles / FEW_S;  // this CTA's 16-row tiles of B
  // This CTA's share of B in pieces.
  const int npieces = (n1 - n0 + 15) / 16;
  auto fetch = [&](int i) {  // by thread 0
    const int r0 = n0 * 16 + i * FEW_PIECE, r1 = min(min(r0 + FEW_PIECE, n1 * 16), a.N);
    const uint32_t bytes = (uint32_t)((r1 - r0) * a.R * 2);
    mbar_arrive_expect_tx(&full[i % P.pieces], bytes);
    bulk_g2s(smem + (size_t)(i % P.pieces) * FEW_PIECE * a.R * 2, B + (int64_t)r0 * a.R, bytes, &full[i % P.pieces]);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < min(P.pieces, npieces); ++i) fetch(i);
  // ---- h = A x. Most groups have few tokens: those take the code for one token tile, whatever the call's size.
  const int wk = 8 / few_wr(a.R), steps = (a.K + 31) / 32;
  const FewGroup G = {A, B, count, n0, n1, s * steps / FEW_S, (s + 1) * steps / FEW_S, cols};
  if (NT == 1 || nt_used == 1)
    few_shrink<1>(a, G, toks, red, P.RP, warp, lane);
  else
    few_shrink<NT>(a, G, toks, red, P.RP, warp, lane);
  __syncthreads();
  const int vals = count * P.RP;
  for (int i = threadIdx.x; i < vals; i += FEW_THREADS) {
    float v = 0.f;
    for (int w = 0; w < wk; ++w) v += red[(size_t)w * cols * P.RP + i];
    part[i] = v;
  }
  cluster_sync();
  {
    const float sc = __ldg(a.scale + ad);
    const uint32_t local = smem_addr(part);
    uint16_t* lo = hs + cols * (P.RP + 8);
    for (int i = threadIdx.x * 4; i < cols * P.RP; i += FEW_THREADS * 4) {
      float4 u[FEW_S];
#pragma unroll
      for (int q = 0; q < FEW_S; ++q)
        u[q] = i < vals ? ld_dsmem_f4(dsmem_addr(local + i * 4, q)) : make_float4(0.f, 0.f, 0.f, 0.f);
      float4 v = u[0];
#pragma unroll
      for (int q = 1; q < FEW_S; ++q) {
        v.x += u[q].x;
        v.y += u[q].y;
        v.z += u[q].z;
        v.w += u[q].w;
      }
      v.x *= sc;
      v.y *= sc;
      v.z *= sc;
      v.w *= sc;
      uint2 hv, lv;
      halves(v, hv, lv);
      const int at = i / P.RP * (P.RP + 8) + i % P.RP;
      *reinterpret_cast<uint2*>(hs + at) = hv;
      *reinterpret_cast<uint2*>(lo + at) = lv;
    }
  }
  cluster_arrive();  // this CTA has read the others' sums
  __syncthreads();
  // ---- rows of B h
  if (NT == 1 || nt_used == 1)
    few_expand<1, STEP>(a, G, toks, smem, hs, P, full, empty, npieces, warp, lane, fetch);
  else
    few_expand<NT, STEP>(a, G, toks, smem, hs, P, full, empty, npieces, warp, lane, fetch);
  cluster_wait();  // the others' shared memory stayed until it had been read
}

}  // namespace lora
}  // namespace flint

using namespace flint;
using namespace flint::lora;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Bytes from the first of `rows` rows (cols bf16 values, ld apart) to the end of the last.
size_t rows_bytes(int64_t ld, int cols, int rows) { return rows == 0 ? 0 : 2 * ((size_t)(rows - 1) * ld + cols); }
bool overlap_bytes(const void* p, size_t np, const void* q, size_t nq) {
  if (!p || !q || np == 0 || nq == 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np;
}
// Whether two sets of rows share memory, by their extents.
bool overlap(const void* p, int64_t ldp, int colsp, const void* q, int64_t ldq, int colsq, int rows) {
  return overlap_bytes(p, rows_bytes(ldp, colsp, rows), q, rows_bytes(ldq, colsq, rows));
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

constexpr int64_t LD_MOST = 0x7fffffff;  // row strides are kept in 32 bits
constexpr int SMALL_T = 32;  // calls of up to this many tokens take the kernels for few rows

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    n = 152;
  return n;
}

// Tiles at most: full ones, and a part-filled one for each group of tokens.
int tiles_most(const flint_lora* l, int T) { return T / TM + std::min(l->num_adapters + 1, T); }

// Tiles of a chunk of the weights' gradients, so that slabs x chunks are about as many CTAs as run at once, two on an
// SM (8192 tokens of 2048 x 2048, rank 32: 62.3 us a call; with three times as many 67.6).
constexpr int DW_CTAS = 152 * 2;
int slabs(const flint_lora* l) { return (l->in_dim + 127) / 128 + (l->out_dim + 127) / 128; }
int chunk_tiles(const flint_lora* l, int T) {
  return std::max(1, (int)(((int64_t)T / TM * slabs(l) + DW_CTAS - 1) / DW_CTAS));
}
// Partial sums are kept for adapters of more than one chunk: those have more than CT 128 tokens, so there are
// m <= T / (128 CT) of them, with at most T / 128 + m tiles and so (T / 128 + m) / CT + m chunks.
int64_t slots_most(const flint_lora* l, int T) {
  const int CT = chunk_tiles(l, T), m = T / (TM * CT);
  return (T / TM + m) / CT + m;
}

struct WsPlan {
  size_t tiles, rowmap, h, g, chunks, of_adapter, part, y32, total;
};
// The workspace of a call of T tokens: a header, then 256-byte aligned regions.
WsPlan ws_plan(const flint_lora* l, int T, bool grad, bool base) {
  WsPlan w = {};
  size_t o = 256;
  if (T <= SMALL_T && !grad) {
    w.y32 = o;  o = ws_align(o + (base ? sizeof(float) * (size_t)T * l->out_dim : 0));
    w.total = o;
    return w;
  }
  const size_t mt = tiles_most(l, T), plane = 2 * mt * TM * l->rank * 2;
  w.tiles = o;   o = ws_align(o + sizeof(int2) * mt);
  w.rowmap = o;  o = ws_align(o + sizeof(int) * mt * TM);
  w.h = o;       o = ws_align(o + plane);
  if (grad) {
    w.g = o;           o = ws_align(o + plane);
    w.chunks = o;      o = ws_align(o + sizeof(int4) * mt);
    w.of_adapter = o;  o = ws_align(o + sizeof(int2) * l->num_adapters);
    w.part = o;        o = ws_align(o + sizeof(float) * (size_t)slots_most(l, T) * l->rank * (l->in_dim + l->out_dim));
  }
  w.total = o;
  return w;
}

// What a workspace for up to T tokens must hold: the partial sums of a shorter call can be more (its chunks are
// shorter), by a count that never passes 3 T / 128, nor 3 DW_CTAS / slabs + 8.
size_t ws_most(const flint_lora* l, int T, bool grad, bool base) {
  size_t most = ws_plan(l, T, grad, base).total;
  if (!grad) return std::max(most, ws_plan(l, std::min(T, SMALL_T), false, base).total);
  const int64_t slots = std::min<int64_t>(3 * (T / TM), 3 * (DW_CTAS / slabs(l)) + 8);
  const int64_t more = slots - slots_most(l, T);
  return most + (more > 0 ? ws_align((size_t)more * sizeof(float) * l->rank * (l->in_dim + l->out_dim)) : 0);
}

FewArgs few_args(const flint_lora* l, const int32_t* adapter, int T) {
  FewArgs p = {};
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

Args tile_args(const flint_lora* l, const int32_t* adapter, int T, uint8_t* ws, const WsPlan& w) {
  Args p = {};
  p.K = l->in_dim;
  p.N = l->out_dim;
  p.R = l->rank;
  p.Rp = (l->rank + 15) & ~15;
  p.n = l->num_adapters;
  p.T = T;
  p.scale = l->scale;
  p.adapter = adapter;
  p.max_tiles = tiles_most(l, T);
  p.hdr = reinterpret_cast<int*>(ws);
  p.tiles = reinterpret_cast<int2*>(ws + w.tiles);
  p.rowmap = reinterpret_cast<int*>(ws + w.rowmap);
  p.h = reinterpret_cast<uint16_t*>(ws + w.h);
  p.CT = 1;
  return p;
}

// A pool [n][rows][cols] in boxes of 64 columns x brows rows of one adapter: what lies past an adapter's rows
// reads as zero, not as the next adapter's.
bool map_pool(CUtensorMap* m, const uint16_t* p, int cols, int rows, int n, int brows) {
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)n};
  const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * rows * 2};
  const cuuint32_t box[3] = {BK, (cuuint32_t)brows, 1};
  return encode_bf16(m, p, 3, dims, strides, box);
}
bool map_low(CUtensorMap* m, const uint16_t* p, int R, int max_tiles) {
  const cuuint64_t dims[2] = {(cuuint64_t)R, (cuuint64_t)2 * max_tiles * TM};
  const cuuint64_t strides[1] = {(cuuint64_t)R * 2};
  const cuuint32_t box[2] = {BK, 64};
  return encode_bf16(m, p, 2, dims, strides, box);
}

// Rows of `cols` bf16 values ld apart, in boxes of bcols x brows.
bool map_rows(CUtensorMap* m, const uint16_t* p, int cols, int ld, int rows, int bcols, int brows) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {(cuuint32_t)bcols, (cuuint32_t)brows};
  return encode_bf16(m, p, 2, dims, strides, box, bcols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

bool make_maps(Maps* m, const flint_lora* l, const Args& p) {
  if (!map_pool(&m->a, l->a, p.K, p.R, p.n, p.Rp) || !map_pool(&m->b, l->b, p.R, p.N, p.n, 64) ||
      !map_low(&m->h, p.h, p.R, p.max_tiles))
    return false;
  m->g = m->dy32 = m->x16 = m->dy16 = m->in = m->out = m->h;
  const int D = p.g ? p.K : p.N;  // columns of the base and output rows
  if (!map_rows(&m->x32, p.x, p.K, p.ldx, p.T, 64, 32)) return false;
  if (p.g && (!map_low(&m->g, p.g, p.R, p.max_tiles) || !map_rows(&m->dy32, p.dy, p.N, p.lddy, p.T, 64, 32) ||
              !map_rows(&m->x16, p.x, p.K, p.ldx, p.T, 64, 16) || !map_rows(&m->dy16, p.dy, p.N, p.lddy, p.T, 64, 16)))
    return false;
  if (p.in && !map_rows(&m->in, p.in, D, p.ldo, p.T, 32, 32)) return false;
  return !p.out || map_rows(&m->out, p.out, D, p.ldo, p.T, 32, 32);
}

// Prepares a kernel once for each device: its dynamic shared memory, and the largest shared-memory carveout, which all
// kernels of a call ask for, because an SM runs blocks of two kernels side by side only under one carveout.
template <typename K>
bool prepare(K kernel, std::atomic<uint64_t>& done, size_t smem) {
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

// A launch that may start while the kernel before it drains (each kernel waits for it itself), in clusters of `cx`.
template <typename... P>
bool launch(void (*kernel)(P...), dim3 grid, int block, size_t smem, int cx, cudaStream_t stream, const P&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cx;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cx > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

std::atomic<uint64_t> g_plan{0}, g_shrink{0}, g_dw_sum{0};

bool run_plan(const Args& p, cudaStream_t stream) {
  return prepare(k_lora_plan, g_plan, plan_smem(FLINT_LORA_MAX_ADAPTERS, PLAN_T)) &&
         launch(k_lora_plan, dim3(1), 1024, plan_smem(p.n, p.T), 0, stream, p);
}

// h (and with `grads` g) of every tile. CTAs of a tile's cluster: as many as run at once, two on an SM, if there were
// all the tiles that T tokens of this pool can make (4096 tokens of 2048 x 2048, 49 tiles at most: 24.9 us a call with
// clusters of 4, 27.2 of 2, 27.7 of 8), and no more than a CTA has k-blocks to take. The host does not know how many
// adapters a batch uses: a large pool leaves room for tiles that are not there, and the clusters are smaller then
// (777 tokens: 8 CTAs with a pool of 16, 2 with 100, 1 from 150 on).
bool run_shrink(const Args& p, const Maps& m, bool grads, cudaStream_t stream) {
  const int kb = (std::min(p.K, grads ? p.N : p.K) + BK - 1) / BK, per = p.max_tiles * (grads ? 2 : 1);
  int S = 1;
  while (S < 8 && per * S * 2 <= 2 * sm_count() && S * 2 <= kb) S *= 2;
  return prepare(k_lora_shrink, g_shrink, shrink_smem(FLINT_LORA_MAX_RANK, true)) &&
         launch(k_lora_shrink, dim3(S, p.max_tiles, grads ? 2 : 1), SHR_THREADS, shrink_smem(p.R, grads), S, stream, p, m);
}

template <bool GRAD, bool WIDE>
bool run_expand_as(const Args& p, const Maps& m, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const int D = GRAD ? p.K : p.N;
  const int64_t items = (int64_t)p.max_tiles * ((D + 127) / 128);
  const size_t smem = exp_smem(p.R);
  return prepare(k_lora_expand<GRAD, WIDE>, done, smem) &&
         launch(k_lora_expand<GRAD, WIDE>, dim3((unsigned)std::min<int64_t>(sm_count(), items)), EXP_THREADS, smem, 0, stream, p, m);
}
template <bool GRAD>
bool run_expand(const Args& p, const Maps& m, cudaStream_t stream) {
  return p.R > 64 ? run_expand_as<GRAD, true>(p, m, stream) : run_expand_as<GRAD, false>(p, m, stream);
}

template <bool WIDE>
bool run_dw(const Args& p, const Maps& m, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  // chunks: the tiles of adapters in runs of CT, and a shorter run for each adapter
  const int chunks = std::min(p.max_tiles, p.max_tiles / p.CT + std::min(p.n, p.T) + 1);
  return prepare(k_lora_dw<WIDE>, done, dw_smem(p.R)) &&
         launch(k_lora_dw<WIDE>, dim3(p.slabs_a + p.slabs_b, chunks), DW_THREADS, dw_smem(p.R), 0, stream, p, m);
}

template <int NT, int STEP>
bool run_few_as(FewArgs p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const int groups = std::min(p.T, p.n + (p.with_none ? 1 : 0)), most = few_pieces(p.N);
  p.smem = std::max(few_plan(p.R, 8 * NT, most, FEW_SMEM).total, few_plan(p.R, 8, most, FEW_SMEM).total);
  return prepare(k_lora_few<NT, STEP>, done, 184 * 1024) &&
         launch(k_lora_few<NT, STEP>, dim3(FEW_S, groups), FEW_THREADS, p.smem, FEW_S, stream, p);
}
bool run_few(const FewArgs& p, cudaStream_t stream) {
  if (p.R % 32 == 0)
    return p.T <= 8 ? run_few_as<1, 32>(p, stream) : p.T <= 16 ? run_few_as<2, 32>(p, stream) : run_few_as<4, 32>(p, stream);
  return p.T <= 8 ? run_few_as<1, 16>(p, stream) : p.T <= 16 ? run_few_as<2, 16>(p, stream) : run_few_as<4, 16>(p, stream);
}

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
  return ws_most(l, max_tokens, false, false);
}

extern "C" size_t flint_gemv_lora_workspace_bytes(const flint_lora* l, int32_t max_batch) {
  if (check_lora(l) != FLINT_MOE_OK || max_batch < 1 || max_batch > MAX_BATCH) return 0;
  return ws_most(l, max_batch, false, true);
}

extern "C" size_t flint_lora_backward_workspace_bytes(const flint_lora* l, int32_t max_tokens) {
  if (check_lora(l) != FLINT_MOE_OK || max_tokens < 1 || max_tokens > FLINT_LORA_MAX_TOKENS) return 0;
  return ws_most(l, max_tokens, true, false);
}

extern "C" flint_moe_status flint_lora_apply(const flint_lora* l, const uint16_t* x, int64_t ldx, const int32_t* adapter,
                                             int32_t T, const uint16_t* y_in, uint16_t* y_out, int64_t ldy, void* ws,
                                             size_t ws_bytes, cudaStream_t stream) {
  const flint_moe_status st = check_pool(l);
  if (st != FLINT_MOE_OK) return st;
  if (T < 0 || T > FLINT_LORA_MAX_TOKENS || ldx < l->in_dim || ldy < l->out_dim || ldx > LD_MOST || ldy > LD_MOST)
    return FLINT_MOE_EINVAL;
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
  uint8_t* wb = static_cast<uint8_t*>(ws);
  if (T <= SMALL_T) {
    FewArgs p = few_args(l, adapter, T);
    p.x = x;
    p.ldx = ldx;
    p.in = y_in;
    p.out = y_out;
    p.ldo = ldy;
    p.with_none = y_in != y_out;
    p.status = reinterpret_cast<int*>(wb) + H_STATUS;
    p.clear = 1;
    return run_few(p, stream) ? FLINT_MOE_OK : FLINT_MOE_ECUDA;
  }
  Args p = tile_args(l, adapter, T, wb, w);
  p.with_none = y_in != y_out;
  p.in = y_in;
  p.out = y_out;
  p.ldo = (int)ldy;
  p.x = x;
  p.ldx = (int)ldx;
  Maps m;
  if (!make_maps(&m, l, p)) return FLINT_MOE_ECUDA;
  return run_plan(p, stream) && run_shrink(p, m, false, stream) && run_expand<false>(p, m, stream) ? FLINT_MOE_OK
                                                                                                   : FLINT_MOE_ECUDA;
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
  FewArgs p = few_args(l, adapter, B);
  p.x = x;
  p.ldx = K;
  p.out32 = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.y32);
  p.status = dev_status ? dev_status : static_cast<int32_t*>(ws) + H_STATUS;
  p.clear = !dev_status;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(packed, 16)) return FLINT_MOE_EALIGN;  // before the first launch
  if (!run_few(p, stream)) return FLINT_MOE_ECUDA;
  return gemv_impl(packed, N, K, fmt, x, B, y, nullptr, 0.f, p.out32, adapter, l->num_adapters, p.status, stream);
}

extern "C" flint_moe_status flint_lora_backward(const flint_lora* l, const uint16_t* x, int64_t ldx, const uint16_t* dy,
                                                int64_t lddy, const int32_t* adapter, int32_t T, const uint16_t* dx_in,
                                                uint16_t* dx_out, int64_t lddx, uint16_t* da, uint16_t* db, void* ws,
                                                size_t ws_bytes, cudaStream_t stream) {
  const flint_moe_status st = check_pool(l);
  if (st != FLINT_MOE_OK) return st;
  if (T < 0 || T > FLINT_LORA_MAX_TOKENS || ldx < l->in_dim || lddy < l->out_dim || ldx > LD_MOST || lddy > LD_MOST ||
      (dx_out && (lddx < l->in_dim || lddx > LD_MOST)))
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
  // the gradients are written while the rows and the adapters are still read
  const size_t na = nw * l->in_dim * 2, nb = nw * l->out_dim * 2;
  const size_t xb = rows_bytes(ldx, l->in_dim, T), yb = rows_bytes(lddy, l->out_dim, T), db_x = rows_bytes(lddx, l->in_dim, T);
  const struct { const void* p; size_t n; } outs[2] = {{da, na}, {db, nb}},
      ins[6] = {{l->a, na}, {l->b, nb}, {x, xb}, {dy, yb}, {dx_in, dx_out ? db_x : 0}, {dx_out, dx_out ? db_x : 0}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (overlap_bytes(o.p, o.n, i.p, i.n)) return FLINT_MOE_EINVAL;
  if (overlap_bytes(da, na, db, nb)) return FLINT_MOE_EINVAL;
  const WsPlan w = ws_plan(l, T, true, false);
  if (ws_bytes < w.total) return FLINT_MOE_EINVAL;
  Args p = tile_args(l, adapter, T, static_cast<uint8_t*>(ws), w);
  p.with_none = dx_out && dx_in != dx_out;
  p.g = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + w.g);
  p.in = dx_out ? dx_in : nullptr;
  p.out = dx_out;
  p.ldo = (int)lddx;
  p.CT = chunk_tiles(l, T);
  p.slabs_a = (p.K + 127) / 128;
  p.slabs_b = (p.N + 127) / 128;
  p.chunks = reinterpret_cast<int4*>(static_cast<uint8_t*>(ws) + w.chunks);
  p.of_adapter = reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + w.of_adapter);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.part);
  p.dA = da;
  p.dB = db;
  p.x = x;
  p.ldx = (int)ldx;
  p.dy = dy;
  p.lddy = (int)lddy;
  Maps m;
  if (!make_maps(&m, l, p)) return FLINT_MOE_ECUDA;
  // The weights' gradients come first after the shrink: x and dy, which both read, may still be in L2 then.
  if (!run_plan(p, stream) || !run_shrink(p, m, true, stream) ||
      !(p.R > 64 ? run_dw<true>(p, m, stream) : run_dw<false>(p, m, stream)) || (dx_out && !run_expand<true>(p, m, stream)))
    return FLINT_MOE_ECUDA;
  const int64_t all = (int64_t)p.R * (p.K + p.N);
  if (!prepare(k_lora_dw_sum, g_dw_sum, 0) ||
      !launch(k_lora_dw_sum, dim3((unsigned)std::min<int64_t>((all + 2047) / 2048, std::max(1, 152 * 8 / p.n)), p.n), 256, 0, 0,
              stream, p))
    return FLINT_MOE_ECUDA;
  return FLINT_MOE_OK;
}
