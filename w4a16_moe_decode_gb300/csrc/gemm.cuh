// Dense matrix products on the 5th-generation tensor cores, with the epilogues of the dense gated feed-forward block
// (ffn.cu) and of the orthogonalised update (orthogonalize.cu) in the same kernel.
//
// D[m][n] = sum_k A[m][k] B[n][k], 16-bit operands (both bf16 or both f16), FP32 sums in tensor memory. Each operand is
// used as it lies in memory: K-major (rows of k) or MN-major (rows of m or n, the reduction being the rows), so that no
// matrix is ever transposed in memory. The reduction may run over several pairs of operands one after the other
// (segments).
#pragma once

#include <algorithm>

#include "tensor.cuh"

namespace flint {
namespace gemm {

constexpr int BK = 64;               // reduction of a stage: one 128-byte swizzled row of 16-bit values
constexpr int BOX = 64 * BK * 2;     // 8 KiB: 64 x 64 values, what one TMA load moves
constexpr int SLOT = 32 * 64;        // 2 KiB: 32 rows x 32 columns of 16-bit values, what one TMA store moves
constexpr int SLOTS = 4;             // of each epilogue warp in k_gemm

// k_gemm: one 128 x 128 tile a CTA, two CTAs on an SM, so that the one's epilogue runs beside the other's products; or
// 128 x 64, whose shorter epilogue counts where the tiles do not fill the card (a 256 x 2048 update, 17 launches: 139 us
// with 128 x 128 tiles, 101). STAGES beside another CTA, DEEP on an SM of its own.
struct One {
  static constexpr int TM = 128, TN = 128, CTAS = 1, STAGES = 3, DEEP = 6, GROUPS = 1, BBOXES = 2;
};
struct Half {
  static constexpr int TM = 128, TN = 64, CTAS = 1, STAGES = 4, DEEP = 8, GROUPS = 1, BBOXES = 1;
};
// k_gemm_pair: 256 x 256 tiles by pairs of CTAs (cta_group::2), each with half of A's rows and half of B's, 128 x 256 sums
// a CTA; persistent, with two accumulators, so that a tile's epilogue runs beside the next one's products. A CTA loads half
// of what it multiplies (32 KB in 512 cycles of MMAs): 8192 tokens of 2048 x 8192 forward, 716 us with one CTA a tile,
// 552. Five stages or six: the same. The last round's tiles split in two to fill it: no gain, since the card's power
// limit lets the busy SMs run faster while others idle. Epilogues that
// read matrices have them brought by TMA, a chunk ahead, in the room of a stage (the gradients' first product, 8192 tokens
// of 2048 x 8192: 309 us with loads by rows).
template <int INS>
struct Pairs {
  static constexpr int TM = 256, TN = 256, CTAS = 2, STAGES = INS ? 4 : 5, GROUPS = 2, BBOXES = 2;
  static constexpr int OUT_SLOTS = INS ? 2 : 4, IN_SLOTS = 2 * INS;  // of each epilogue warp
};
using Two = Pairs<0>;  // (the tiles are the same)
// A CTA's operands of a stage: 128 x 64 of A, 64 BBOXES x 64 of B.
template <typename C>
constexpr int STAGE = (2 + C::BBOXES) * BOX;
// Epilogue warps come in GROUPS of four (tensor memory's lanes), 128 of the accumulator's columns each.
template <typename C>
constexpr int THREADS = 64 + 128 * C::GROUPS;  // warp 0 loads, warp 1 issues the MMAs, the others the epilogue
template <typename C>
constexpr size_t SMEM = 1024 + (size_t)C::DEEP * STAGE<C>;
template <typename C>
constexpr size_t PAIR_SMEM = 1024 + (size_t)C::STAGES * STAGE<C> + (size_t)C::GROUPS * 4 * (C::OUT_SLOTS + C::IN_SLOTS) * SLOT;
static_assert(PAIR_SMEM<Pairs<0>> <= 227 * 1024 - 512 && PAIR_SMEM<Pairs<2>> <= 227 * 1024 - 512, "shared memory of a CTA");
static_assert(4 * SLOTS * SLOT + One::TM * One::TN * 4 <= One::STAGES * STAGE<One> && Half::STAGES * STAGE<Half> == One::STAGES * STAGE<One>,
              "k_gemm's epilogue writes where its operands were");

constexpr int MOST = 4;        // products of one launch
constexpr int DEEP_FROM = 40;  // k-blocks of a CTA from which it takes all of its SM's memory

struct Problem {
  int M, N;         // output rows and columns (of one matrix of the batch)
  int kb;           // k-blocks of a segment
  int segs;         // segments: products of the operands' matrices that the masks' bits name, added up
  int a_of, b_of;
  int a_mn, b_mn;   // operands stored MN-major
  int sym;          // D is its own transpose: the tiles above the diagonal are computed, and written twice
  int batch;
  // Operands (1: A, 2: B) that k_gemm asks for without waiting for the launch before: what neither that launch writes nor
  // anything before it still does, since that launch lets this one begin only after its own wait.
  int early;
  __host__ __device__ int blocks() const { return kb * segs; }
};
struct Args {
  Problem p[MOST];
  int n;            // of them
  int f16;          // operands are f16, not bf16
  int* status;
  int clear;        // the first kernel of a call clears the status word
};

// Operands in 64 x 64 boxes (x: the contiguous dimension, y: rows, z: matrix of the batch); what an epilogue writes and,
// behind that, what it reads in 32 x 32 boxes.
template <int IO>
struct Maps {
  CUtensorMap a[2], b[2];
  CUtensorMap io[IO];
};
// An epilogue E has OUTS and INS of them, for each of up to MAPS products of a launch. PAIR: its columns are two products'
// (B has two operands). SMALL: its matrices have one tile of 64 columns at most, which k_gemm alone is for.
template <typename E>
using MapsOf = Maps<E::OUTS + E::INS>;
template <int IO, int N>
struct MapSet {
  Maps<IO> of[N];
};
template <typename E>
using AllMaps = MapSet<E::OUTS + E::INS, E::MAPS>;

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

__device__ __forceinline__ uint32_t f2b2(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint4 pack8_bf16(const float* v) {
  return make_uint4(f2b2(v[0], v[1]), f2b2(v[2], v[3]), f2b2(v[4], v[5]), f2b2(v[6], v[7]));
}
__device__ __forceinline__ void unpack8_bf16(const uint4 u, float* v) {
  v[0] = bf16lo(u.x), v[1] = bf16hi(u.x), v[2] = bf16lo(u.y), v[3] = bf16hi(u.y);
  v[4] = bf16lo(u.z), v[5] = bf16hi(u.z), v[6] = bf16lo(u.w), v[7] = bf16hi(u.w);
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// What an epilogue warp works on: 32 rows, a lane each.
struct Part {
  int row0, row;  // the warp's first output row, and this lane's
  int n0;         // the tile's first output column
  int z, M, N;
  bool twice;     // the transposed place gets the same values
  int lane;
  uint8_t* sm;    // the warp's slots
  uint32_t sm_addr;
  int slot, slots;  // the next one to fill, of how many
  float4 f;         // what the epilogue keeps of its matrix (E::matrix, once a tile)

  // The place of 16-byte piece c of this lane's row in a slot: the 64-byte swizzle.
  static __device__ __forceinline__ uint32_t piece(int lane, int c) { return (uint32_t)(lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)); }
  __device__ __forceinline__ void begin() const {
    if (lane == 0) {
      if (slots == 4)
        bulk_wait_read<3>();
      else
        bulk_wait_read<1>();
    }
    __syncwarp();
  }
  __device__ __forceinline__ void end(const CUtensorMap* map, int x, int y, bool in) {
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      if (in) tma_store_3d(map, x, y, z, sm_addr + slot * SLOT);
      bulk_commit();
    }
    slot = slot + 1 == slots ? 0 : slot + 1;
  }
  // 32 columns x .. of the warp's rows, this lane's row in v: to the next slot, and from there to memory (what lies
  // outside the matrix is left out).
  __device__ __forceinline__ void put(const CUtensorMap* map, int x, const uint4 (&v)[4]) {
    begin();
#pragma unroll
    for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(sm + slot * SLOT + piece(lane, c)) = v[c];
    end(map, x, row0, x < N && row0 < M);
  }
  // The same values as columns row0 .. of rows x ..
  __device__ __forceinline__ void put_transposed(const CUtensorMap* map, int x, const uint4 (&v)[4]) {
    begin();
    uint8_t* s = sm + slot * SLOT + (lane & 7) * 2;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const uint4& u = v[c >> 3];
      const uint32_t w = (c & 6) == 0 ? u.x : (c & 6) == 2 ? u.y : (c & 6) == 4 ? u.z : u.w;
      *reinterpret_cast<uint16_t*>(s + c * 64 + ((((lane >> 3) ^ (c >> 1)) & 3) << 4)) = (uint16_t)(c & 1 ? w >> 16 : w);
    }
    end(map, row0, x, x < N && row0 < M);
  }
};

// Nothing read beside the sums.
struct NoPre {
  template <typename A>
  __device__ __forceinline__ NoPre(const A&, const Part&, int) {}
  __device__ __forceinline__ NoPre(const Part&, const uint8_t*) {}
};
// This lane's row of an input slot.
__device__ __forceinline__ void slot_row(const Part& t, const uint8_t* in, uint4 (&v)[4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] = lds128(in + Part::piece(t.lane, c));
}

// Tiles of a launch: its products one after the other, each batch of one in bands of eight rows of tiles, column by
// column, so that the tiles that run at once share their operands in L2; above the diagonal only, row by row, where the
// result is its own transpose.
template <typename C, bool PAIR>
struct Walk {
  static constexpr int COLS = PAIR ? C::TN / 2 : C::TN;
  __host__ __device__ static int down(const Problem& p) { return (p.M + C::TM - 1) / C::TM; }
  __host__ __device__ static int across(const Problem& p) { return (p.N + COLS - 1) / COLS; }
  __host__ __device__ static int each(const Problem& p) { return p.sym ? down(p) * (down(p) + 1) / 2 : down(p) * across(p); }
  __host__ __device__ static int64_t tiles(const Args& a) {
    int64_t t = 0;
    for (int i = 0; i < a.n; ++i) t += (int64_t)each(a.p[i]) * a.p[i].batch;
    return t;
  }
  int i, m, n, z;  // product, tile and matrix of it
  __device__ __forceinline__ Walk(const Args& a, int t) {
    i = 0;
    int per = each(a.p[0]);
    if constexpr (!PAIR)
      while (i + 1 < a.n && t >= per * a.p[i].batch) {
        t -= per * a.p[i].batch;
        per = each(a.p[++i]);
      }
    const Problem& p = a.p[i];
    const int mt = down(p), nt = across(p);
    z = t / per;
    t -= z * per;
    if (p.sym) {
      for (m = 0; t >= mt - m; ++m) t -= mt - m;
      n = m + t;
    } else {
      const int band = t / (8 * nt), first = band * 8, rows = min(8, mt - first);
      t -= band * 8 * nt;
      n = t / rows;
      m = first + t - n * rows;
    }
  }
};

// Descriptors of one operand of a stage (128 rows or columns x 64 of the reduction).
struct Operand {
  uint64_t desc;  // without the address
  uint32_t step;  // 16 of the reduction further
  // A CTA of a cluster finds its rank in the upper bits of its shared-memory addresses: they are not the descriptor's.
  __device__ __forceinline__ uint64_t at(uint32_t saddr) const { return desc | ((saddr & 0x3FFFFu) >> 4); }
};
__device__ __forceinline__ Operand operand(bool mn) {
  return mn ? Operand{sw128_desc_mn(0, BOX), 2048 >> 4} : Operand{sw128_desc(0), 32 >> 4};
}

// This CTA's share of a stage: rows m, m + 64 of A and n[0], n[1] of B from k on, by one thread.
template <typename C, typename Load>
__device__ __forceinline__ void load_stage(bool a_mn, bool b_mn, int k, int m, const int (&n)[2], Load load) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int mm = m + 64 * h;
    load(h * BOX, true, h, a_mn ? mm : k, a_mn ? k : mm);
    if (h < C::BBOXES) load((2 + h) * BOX, false, h, b_mn ? n[h] : k, b_mn ? k : n[h]);
  }
}

__device__ __forceinline__ uint32_t idesc_of(const Args& a, const Problem& p, int m, int n) {
  return idesc_f32acc(m, n, !a.f16) | (p.a_mn ? IDESC_A_MN : 0u) | (p.b_mn ? IDESC_B_MN : 0u);
}

// One tile a CTA, or a cluster of S = 2, 4 or 8 CTAs a tile, each with a run of the k-blocks: their sums meet in
// distributed shared memory, 32 x 32 blocks of the tile shared out among the CTAs' epilogue warps, which add them in CTA
// order from their own CTA on (so that no CTA's memory is asked by all at once).
template <typename C, typename E, int ST>
__global__ void __launch_bounds__(THREADS<C>, 2) k_gemm(const Args a, const __grid_constant__ AllMaps<E> all, const typename E::Args e) {
  extern __shared__ uint8_t dsmem[];
  __shared__ uint64_t full[ST], empty[ST], acc_full;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_addr(dsmem) + 1023u) & ~1023u;
  volatile int* abort = &abort_flag;
  if (threadIdx.x < ST) {
    mbar_init(&full[threadIdx.x], 1);
    mbar_init(&empty[threadIdx.x], 1);
    if (threadIdx.x == 0) {
      mbar_init(&acc_full, 1);
      abort_flag = 0;
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base, C::TN);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  // (x: the CTAs of a tile, y: tiles)
  const int S = gridDim.x, rank = blockIdx.x;
  const Walk<C, E::PAIR> w(a, blockIdx.y);
  const Problem& p = a.p[w.i];
  const MapsOf<E>& maps = all.of[w.i];
  if (threadIdx.x == 0) {
    prefetch_map(&maps.a[0]);
    prefetch_map(&maps.b[0]);
    prefetch_map(&maps.io[0]);
  }
  const int blocks = p.blocks(), b0 = blocks * rank / S, b1 = blocks * (rank + 1) / S;
  const int m0 = w.m * C::TM, n0 = w.n * w.COLS;
  if (warp != 0) {
    pdl_wait();
    pdl_trigger();
    if (a.clear && warp == 1 && lane == 0 && blockIdx.x + blockIdx.y == 0) *a.status = 0;
  }
  if (warp == 0) {
    if (lane == 0) {
      const int n[2] = {n0, E::PAIR ? n0 : n0 + 64};
      const bool a_mn = p.a_mn, b_mn = p.b_mn;
      // Boxes that lie outside the matrix are not asked for: the rows and columns that come of them are not read.
      const bool a_both = m0 + 64 < p.M, b_both = C::BBOXES == 2 && (E::PAIR || n[1] < p.N);
      const uint32_t bytes = (2 + (a_both ? 1 : 0) + (b_both ? 1 : 0)) * BOX;
      const int per = p.kb;
      // The stages that need not wait for room: at first the operands that are there already, then the others.
      const int n_blocks = b1 - b0, stages = min(ST, n_blocks);
      int i = 0, s = 0, seg = 0, kb = 0;
      uint32_t phase = 0;
      const CUtensorMap *am = nullptr, *bm = nullptr;
      auto begin = [&] {
        i = 0, s = 0;
        seg = b0 / per, kb = b0 - seg * per;
        am = &maps.a[(p.a_of >> seg) & 1], bm = &maps.b[(p.b_of >> seg) & 1];
      };
      auto next = [&] {
        ++i;
        if (++kb == per) {
          kb = 0;
          ++seg;
          am = &maps.a[(p.a_of >> seg) & 1], bm = &maps.b[(p.b_of >> seg) & 1];
        }
        if (++s == ST) s = 0, phase ^= 1;
      };
      auto load = [&](bool with_a, bool with_b) {
        const uint32_t sm = base + s * STAGE<C>;
        load_stage<C>(a_mn, b_mn, kb * BK, m0, n, [&](int off, bool is_a, int h, int x, int y) {
          if (is_a ? with_a && (h == 0 || a_both) : with_b && (h == 0 || b_both))
            tma_load_3d(sm + off, is_a ? am : E::PAIR ? &maps.b[h] : bm, x, y, w.z, &full[s]);
        });
      };
      for (begin(); i < stages; next()) {
        mbar_arrive_expect_tx(&full[s], bytes);
        load(p.early & 1, p.early & 2);
      }
      pdl_wait();
      pdl_trigger();
      phase = 0;
      for (begin(); i < stages; next()) load(!(p.early & 1), !(p.early & 2));
      for (; i < n_blocks; next()) {
        if (!wait_ab(&empty[s], phase ^ 1, abort, a.status)) break;
        mbar_arrive_expect_tx(&full[s], bytes);
        load(true, true);
      }
      for (int r = (i > ST ? i - ST : 0); r < i; ++r) mbar_drain(&full[r % ST], (r / ST) & 1);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_of(a, p, C::TM, C::TN);
    const Operand oa = operand(p.a_mn), ob = operand(p.b_mn);
    int i = 0, s = 0;
    uint32_t phase = 0;
    for (; i < b1 - b0; ++i) {
      const bool ok = wait_ab(&full[s], phase, abort, a.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t ad = oa.at(base + s * STAGE<C>), bd = ob.at(base + s * STAGE<C> + 2 * BOX);
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks) tc_mma(tmem, ad + ks * oa.step, bd + ks * ob.step, idesc, (i > 0 || ks > 0) ? 1u : 0u);
        tc_commit(&empty[s]);
        if (i + 1 == b1 - b0) tc_commit(&acc_full);
      }
      __syncwarp();
      if (++s == ST) s = 0, phase ^= 1;
    }
    for (int r = (i > ST ? i - ST : 0); r < i; ++r) mbar_drain(&empty[r % ST], (r / ST) & 1);
  }
  // The epilogue's warps: slots and partial sums lie where the operands were.
  const int q = warp & 3;
  uint32_t w1[32], w2[32];
  Part t;
  t.n0 = n0;
  t.z = w.z;
  t.M = p.M;
  t.N = p.N;
  t.twice = p.sym && w.m != w.n;
  t.lane = lane;
  t.sm_addr = base + q * SLOTS * SLOT;
  t.sm = dsmem + (t.sm_addr - smem_addr(dsmem));
  t.slot = 0;
  t.slots = SLOTS;
  constexpr int CHUNKS = Walk<C, E::PAIR>::COLS / 32;
  if (warp >= 2) {
    E::matrix(e, t);
    const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16);
    if (S == 1) {
      t.row0 = m0 + q * 32;
      t.row = t.row0 + lane;
      typename E::Pre pre(e, t, 0);  // what a chunk reads besides the sums is asked for a chunk ahead
      if (__all_sync(0xffffffffu, wait_ab(&acc_full, 0, abort, a.status)) && t.row0 < t.M) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < w.COLS; c += 32) {
          tc_ld32_async(acc + c, w1);
          if constexpr (E::PAIR) tc_ld32_async(acc + C::TN / 2 + c, w2);
          const typename E::Pre now = pre;
          if (c + 32 < w.COLS) pre = typename E::Pre(e, t, c + 32);
          tc_wait_ld();
          E::chunk(e, maps, t, c, w1, w2, now);
        }
      }
    } else if (__all_sync(0xffffffffu, wait_ab(&acc_full, 0, abort, a.status))) {
      tc_fence_after();
      // Row r's four columns 4 c .. at piece c * 128 + r, behind the slots.
      float4* part = reinterpret_cast<float4*>(dsmem + (base - smem_addr(dsmem)) + 4 * SLOTS * SLOT) + q * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < C::TN; c += 32) {
        tc_ld32_async(acc + c, w1);
        tc_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          part[(c / 4 + j) * 128] = make_float4(__uint_as_float(w1[4 * j]), __uint_as_float(w1[4 * j + 1]),
                                                __uint_as_float(w1[4 * j + 2]), __uint_as_float(w1[4 * j + 3]));
      }
    }
    tc_fence_before();
  }
  if (S > 1) {
    __syncwarp();
    cluster_sync();
    if (warp >= 2) {
      const uint32_t part = base + 4 * SLOTS * SLOT;
#pragma unroll 1
      for (int u = rank * 4 + q; u < 4 * CHUNKS; u += 4 * S) {  // block u of the tile: rows 32 (u % 4), columns 32 (u / 4)
        t.row0 = m0 + (u & 3) * 32;
        t.row = t.row0 + lane;
        if (t.row0 >= t.M) continue;
        const int c = (u >> 2) * 32;
        const typename E::Pre pre(e, t, c);
        auto sums = [&](int col, uint32_t (&v)[32]) {
          float acc[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[j] = 0.f;
#pragma unroll 1
          for (int r = 0; r < S; ++r) {
            const uint32_t at = dsmem_addr(part + (uint32_t)((col / 4 * 128 + (u & 3) * 32 + lane) * 16), (rank + r) & (S - 1));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 f = ld_dsmem_f4(at + j * 2048);
              acc[4 * j] += f.x, acc[4 * j + 1] += f.y, acc[4 * j + 2] += f.z, acc[4 * j + 3] += f.w;
            }
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(acc[j]);
        };
        sums(c, w1);
        if constexpr (E::PAIR) sums(C::TN / 2 + c, w2);
        E::chunk(e, maps, t, c, w1, w2, pre);
      }
    }
    __syncwarp();
    cluster_sync();  // the other CTAs have read this one's sums
  }
  if (warp >= 2 && lane == 0) bulk_wait_read<0>();  // (the memory that the stores read; they are done when the grid is)
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, C::TN);
  }
}

// ---------------------------------------------------------------------------
// Pairs of CTAs. Each loads its own halves of the operands; all copies arrive on the first CTA's barriers, whose MMA warp
// multiplies for both and tells both when a stage or a tile's sums are done.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives once on bar in both CTAs when every tcgen05 operation this thread issued so far has completed.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <typename E>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS<Two>, 1)
    k_gemm_pair(const Args a, const __grid_constant__ AllMaps<E> all, const typename E::Args e) {
  extern __shared__ uint8_t dsmem[];
  using C = Pairs<E::INS>;
  constexpr int ST = C::STAGES, EPI = 4 * C::GROUPS;
  __shared__ uint64_t full[ST], empty[ST], acc_full[2], acc_empty[2];
  __shared__ uint64_t in_full[EPI][2];  // a warp's input slots filled
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t base = (smem_addr(dsmem) + 1023u) & ~1023u;
  volatile int* abort = &abort_flag;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * EPI);
    }
    if (E::INS)
      for (int w = 0; w < EPI; ++w)
        for (int b = 0; b < 2; ++b) mbar_init(&in_full[w][b], 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(&tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  pdl_wait();
  pdl_trigger();
  if (a.clear && threadIdx.x == 0 && blockIdx.x == 0) *a.status = 0;
  using W = Walk<Two, E::PAIR>;
  const int step = gridDim.x >> 1, first = blockIdx.x >> 1, tiles = (int)W::tiles(a);
  if (warp == 0) {
    if (lane == 0) {
      int i = 0, s = 0;  // stages so far, the next one's place
      uint32_t phase = 0;
      const uint32_t bar0 = dsmem_addr(smem_addr(full), 0);
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        const W w(a, t);
        const Problem& p = a.p[w.i];
        const MapsOf<E>& maps = all.of[w.i];
        // The first CTA holds the first half of the tile's columns of B (or the gate's rows), the second the others.
        const int m = w.m * Two::TM + (int)rank * 128, nb = w.n * W::COLS + (E::PAIR ? 0 : (int)rank * 128);
        const int n[2] = {nb, nb + 64}, per = p.kb;
        const bool a_mn = p.a_mn, b_mn = p.b_mn;
        for (int seg = 0; seg < p.segs && ok; ++seg) {
          const CUtensorMap *am = &maps.a[(p.a_of >> seg) & 1], *bm = &maps.b[E::PAIR ? rank : (p.b_of >> seg) & 1];
          for (int kb = 0; kb < per; ++kb) {
            if (i >= ST && !(ok = wait_ab(&empty[s], phase ^ 1, abort, a.status))) break;
            const uint32_t sm = base + s * STAGE<Two>, bar = bar0 + s * 8;
            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * STAGE<Two>);
            load_stage<Two>(a_mn, b_mn, kb * BK, m, n,
                            [&](int off, bool is_a, int, int x, int y) { tma_load_3d_pair(sm + off, is_a ? am : bm, x, y, w.z, bar); });
            ++i;
            if (++s == ST) s = 0, phase ^= 1;
          }
        }
      }
      // The second CTA's copies count on the first's barriers: it stays until the first has seen them (cluster_sync).
      if (rank == 0)
        for (int r = (i > ST ? i - ST : 0); r < i; ++r) mbar_drain(&full[r % ST], (r / ST) & 1);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      int i = 0, n = 0, s = 0;  // stages and tiles so far, the next stage's place
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step, ++n) {
        const W w(a, t);
        const Problem& p = a.p[w.i];
        const uint32_t idesc = idesc_of(a, p, Two::TM, Two::TN);
        const Operand oa = operand(p.a_mn), ob = operand(p.b_mn);
        const int blocks = p.blocks();
        const int b = n & 1;
        ok = n < 2 || wait_ab(&acc_empty[b], ((n >> 1) - 1) & 1, abort, a.status);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        for (int kb = 0; kb < blocks; ++kb, ++i) {
          ok = wait_ab(&full[s], phase, abort, a.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = oa.at(base + s * STAGE<Two>), bd = ob.at(base + s * STAGE<Two> + 2 * BOX);
#pragma unroll
            for (int ks = 0; ks < BK / 16; ++ks)
              tc_mma_pair(tmem + b * Two::TN, ad + ks * oa.step, bd + ks * ob.step, idesc, (kb > 0 || ks > 0) ? 1u : 0u);
            tc_commit_pair(&empty[s]);
            if (kb + 1 == blocks) tc_commit_pair(&acc_full[b]);
          }
          __syncwarp();
          if (++s == ST) s = 0, phase ^= 1;
        }
      }
      for (int r = (i > ST ? i - ST : 0); r < i; ++r) mbar_drain(&empty[r % ST], (r / ST) & 1);
    }
  } else {
    const int q = warp & 3, group = (warp - 2) >> 2;
    constexpr int each = W::COLS / C::GROUPS;  // columns of a tile for this warp's group
    Part t;
    t.lane = lane;
    t.sm_addr = base + ST * STAGE<Two> + (uint32_t)((warp - 2) * (C::OUT_SLOTS + C::IN_SLOTS) * SLOT);
    t.sm = dsmem + (t.sm_addr - smem_addr(dsmem));
    t.slot = 0;
    t.slots = C::OUT_SLOTS;
    const uint32_t in_addr = t.sm_addr + C::OUT_SLOTS * SLOT;
    const uint8_t* const in_sm = t.sm + C::OUT_SLOTS * SLOT;
    int fetched = 0, used = 0;  // chunks
    // What the epilogue reads beside the sums for the chunk at column c of tile `w`.
    auto fetch = [&](const W& w, int c) {
      if constexpr (E::INS > 0) {
        const int row0 = w.m * Two::TM + (int)rank * 128 + q * 32;
        if (row0 >= a.p[w.i].M) return;
        if (lane == 0) {
          const int b = fetched & 1;
          mbar_arrive_expect_tx(&in_full[warp - 2][b], E::INS * SLOT);
          for (int i = 0; i < E::INS; ++i)
            tma_load_3d(in_addr + (b * E::INS + i) * SLOT, &all.of[w.i].io[E::OUTS + i], w.n * W::COLS + c, row0, w.z, &in_full[warp - 2][b]);
        }
        ++fetched;
      }
    };
    uint32_t w1[32], w2[32];
    int n = 0;
    bool ok = true;
    if (first < tiles) fetch(W(a, first), group * each);
    for (int ti = first; ti < tiles; ti += step, ++n) {
      const int b = n & 1;
      const W w(a, ti);
      const Problem& p = a.p[w.i];
      t.z = w.z;
      t.M = p.M;
      t.N = p.N;
      t.n0 = w.n * W::COLS;
      t.row0 = w.m * Two::TM + (int)rank * 128 + q * 32;
      t.row = t.row0 + lane;
      t.twice = p.sym && w.m != w.n;
      E::matrix(e, t);
      ok = __all_sync(0xffffffffu, wait_ab(&acc_full[b], (n >> 1) & 1, abort, a.status));
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + b * Two::TN + ((uint32_t)(q * 32) << 16);
      const bool live = t.row0 < t.M;
#pragma unroll 1
      for (int c = group * each; c < (group + 1) * each; c += 32) {
        const bool last = c + 32 == (group + 1) * each;
        if (live) {
          tc_ld32_async(acc + c, w1);
          if constexpr (E::PAIR) tc_ld32_async(acc + Two::TN / 2 + c, w2);
        }
        tc_wait_ld();
        if (last) {  // this warp has read the accumulator
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(dsmem_addr(smem_addr(&acc_empty[b]), 0));
        }
        // The next chunk's into the other slots, which all lanes have read.
        if (E::INS) {
          __syncwarp();
          if (!last)
            fetch(w, c + 32);
          else if (ti + step < tiles)
            fetch(W(a, ti + step), group * each);
        }
        if (live) {
          if (E::INS) {
            ok = __all_sync(0xffffffffu, wait_ab(&in_full[warp - 2][used & 1], (used >> 1) & 1, abort, a.status));
            if (!ok) break;
          }
          const typename E::Pre pre(t, in_sm + (used & 1) * E::INS * SLOT);
          if (E::INS) fence_proxy_async();  // these reads come before the copies into the slots
          E::chunk(e, all.of[w.i], t, c, w1, w2, pre);
          ++used;
        }
      }
      if (!ok) break;
    }
    if (E::INS && lane == 0)  // after a failed wait: copies still on their way
      for (; used < fetched; ++used) mbar_drain(&in_full[warp - 2][used & 1], (used >> 1) & 1);
    if (lane == 0) bulk_wait_read<0>();  // (the memory that the stores read; they are done when the grid is)
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing of the other CTA's still counts on this one's barriers or reads its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_free_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// A batch of matrices [rows][cols] of 16-bit values (rows ld apart, matrices `apart`), as an operand or as an output.
inline bool map_matrix(CUtensorMap* m, const void* p, int64_t cols, int64_t rows, int64_t ld, int64_t batch, int64_t apart, bool out) {
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)apart * 2};
  const cuuint32_t side = out ? 32 : 64, box[3] = {side, side, 1};
  return encode_bf16(m, p, 3, dims, strides, box, out ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                     out ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}
inline bool map_in(CUtensorMap* m, const void* p, int64_t cols, int64_t rows, int64_t ld) {
  return map_matrix(m, p, cols, rows, ld, 1, ld, false);  // one matrix: its distance to the next is never used
}
inline bool map_out(CUtensorMap* m, const void* p, int64_t cols, int64_t rows, int64_t ld) {
  return map_matrix(m, p, cols, rows, ld, 1, ld, true);
}

// Prepares a kernel once for each device: its dynamic shared memory, and the carveout that all kernels here ask for.
template <auto KERNEL>
bool prepare(size_t smem) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev > 63) return false;
  if ((done.load() >> dev) & 1) return true;
  if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared) !=
          cudaSuccess ||
      cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return false;
  done.fetch_or((uint64_t)1 << dev);
  return true;
}

// A launch that may start while the kernel before it drains (each kernel waits for it itself), in clusters of `cx`.
template <auto KERNEL, size_t MOST_SMEM, typename... P>
bool launch(dim3 grid, int block, size_t smem, int cx, cudaStream_t stream, const P&... args) {
  if (!prepare<KERNEL>(MOST_SMEM)) return false;
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
  return cudaLaunchKernelEx(&cfg, KERNEL, args...) == cudaSuccess;
}

// SMs of the current device, asked for once.
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev > 63) return 152;
  if ((n = known[dev].load()) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 2) return 152;
  known[dev].store(n);
  return n;
}

// How a launch's products are computed: by pairs of CTAs, or by S CTAs a tile of 128 x 128 or 128 x 64.
struct Choice {
  int kind;  // 0: pairs, 1: 128 x 128 tiles, 2: 128 x 64
  int S;
};
// The same products with all their tiles.
inline Args whole(Args a) {
  for (int i = 0; i < a.n; ++i) a.p[i].sym = 0;
  return a;
}
// The one with the fewest cycles by this estimate (from the times of products of 32 to 8192 rows): a k-block takes pairs
// 600 cycles, a CTA alone on its SM 450 (300 with 64 columns; memory's latency over the stages in flight: with many stages
// 320 and 220), two on an SM 850 (500) together; a tile at least its epilogue's 4000; beginning and end take 9000, 6500
// (5000), half of them again for a tile that others follow, sums over a cluster 3000 more. A launch takes as long as its
// longest tile, or as many rounds of the mean one as it has.
template <typename E>
Choice choose(const Args& a, int64_t* cycles = nullptr) {
  const int64_t sms = sm_count() & ~1;
  Choice best = {0, 1};
  int64_t cost = INT64_MAX;
  auto deep = [&](int per, int64_t slots) { return slots == sms && per >= DEEP_FROM; };
  auto consider = [&](int kind, int S, int64_t slots, const Args& p, auto tiles, int block, int ends) {
    int64_t work = 0, longest = 0, n = 0;
    for (int i = 0; i < p.n; ++i) {
      const int per = (p.p[i].blocks() + S - 1) / S;
      const int64_t t = std::max<int64_t>((int64_t)per * (deep(per, slots) ? block * 7 / 10 : block), 4000) + (slots > sms ? ends / 2 : 0);
      const int64_t m = (int64_t)tiles(p.p[i]) * p.p[i].batch * S;
      work += m * t;
      n += m;
      longest = std::max(longest, t);
    }
    const int64_t rounds = (n + slots - 1) / slots;
    const int64_t c = std::max(longest, work / n * rounds) + ends + (S > 1 ? 3000 : 0);
    if (c < cost) cost = c, best = {kind, S};
  };
  if constexpr (!E::SMALL) consider(0, 1, sms / 2, a, Walk<Two, E::PAIR>::each, 600, 9000);
  int64_t least = 1 << 30;
  for (int i = 0; i < a.n; ++i) least = std::min<int64_t>(least, a.p[i].blocks());
  auto narrow = [&](int kind, const Args& p, int64_t n, auto tiles, int alone, int two, int ends) {
    for (int S = 1; S <= 8 && n <= 65535; S *= 2) {  // (a grid's second dimension)
      if (S > 1 && (n * S > sms || 4 * S > least)) break;
      consider(kind, S, n * S <= sms ? sms : 2 * sms, p, tiles, n * S <= sms ? alone : two, ends);
    }
  };
  if constexpr (!E::SMALL) narrow(1, a, Walk<One, E::PAIR>::tiles(a), Walk<One, E::PAIR>::each, 450, 850, 6500);
  if constexpr (!E::PAIR) narrow(2, whole(a), Walk<Half, false>::tiles(whole(a)), Walk<Half, false>::each, 300, 500, 5000);
  if (cycles) *cycles = cost;
  return best;
}

// k_gemm on S CTAs a tile. Its CTAs take an SM's whole memory for their stages where they have one each and many k-blocks
// (the second product of 1024 tokens of 2048 x 8192, 128 each: 102 -> 90 us a call); with fewer, room for the next launch's
// CTAs to begin in counts more (77 tokens, 16 and 32: 35 us, and 42 with all the memory).
template <typename C, typename E>
bool run_tiles(const Args& a, const AllMaps<E>& m, const typename E::Args& e, int S, cudaStream_t stream) {
  const int64_t tiles = Walk<C, E::PAIR>::tiles(a);
  int most = 0;
  for (int i = 0; i < a.n; ++i) most = std::max(most, (a.p[i].blocks() + S - 1) / S);
  const dim3 grid(S, (unsigned)tiles);
  if (tiles * S <= sm_count() && most >= DEEP_FROM)
    return launch<k_gemm<C, E, C::DEEP>, SMEM<C>>(grid, THREADS<C>, SMEM<C>, S, stream, a, m, e);
  constexpr size_t smem = 1024 + (size_t)C::STAGES * STAGE<C>;
  return launch<k_gemm<C, E, C::STAGES>, smem>(grid, THREADS<C>, smem, S, stream, a, m, e);
}

template <typename E>
bool run(const Args& a, const AllMaps<E>& m, const typename E::Args& e, cudaStream_t stream, const Choice& c) {
  if constexpr (!E::PAIR)
    if (E::SMALL || c.kind == 2) return run_tiles<Half, E>(whole(a), m, e, c.S, stream);
  if constexpr (!E::SMALL) {
    if (c.kind == 1) return run_tiles<One, E>(a, m, e, c.S, stream);
    const int64_t pairs = std::min<int64_t>(Walk<Two, E::PAIR>::tiles(a), sm_count() / 2);
    return launch<k_gemm_pair<E>, PAIR_SMEM<Pairs<E::INS>>>(dim3(2 * (unsigned)pairs), THREADS<Two>, PAIR_SMEM<Pairs<E::INS>>, 0, stream, a, m, e);
  }
}
template <typename E>
bool run(const Args& a, const AllMaps<E>& m, const typename E::Args& e, cudaStream_t stream) {
  return run<E>(a, m, e, stream, choose<E>(a));
}

}  // namespace gemm
}  // namespace flint
