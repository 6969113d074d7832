// Dense matrix products on the 5th-generation tensor cores, with the epilogues of the dense gated feed-forward block
// (ffn.cu) and of the orthogonalised update (orthogonalize.cu) in the same kernel.
//
// D[m][n] = sum_k A[m][k] B[n][k], 16-bit operands (both bf16 or both f16), FP32 sums in tensor memory. Each operand is
// used as it lies in memory: K-major (rows of k) or MN-major (rows of m or n, the reduction being the rows), so that no
// matrix is ever transposed in memory. The reduction may run over two pairs of operands one after the other (segments).
#pragma once

#include <algorithm>

#include "tensor.cuh"

namespace flint {
namespace gemm {

constexpr int TILE = 128;               // rows and columns of an output tile
constexpr int BK = 64;                  // reduction of a stage: one 128-byte swizzled row of 16-bit values
constexpr int BOX = 64 * BK * 2;        // 8 KiB: 64 x 64 values, what one TMA load moves
constexpr int STAGE = 4 * BOX;          // 128 x 64 of A, 128 x 64 of B
constexpr int STAGES = 3;
constexpr int THREADS = 192;            // warp 0 loads, warp 1 issues the MMAs, warps 2-5 the epilogue
constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE;

struct Args {
  int M, N;        // output rows and columns (of one matrix of the batch)
  int kb[2];       // k-blocks of the two segments (0: no second segment)
  int* status;
  int clear;       // the first kernel of a call clears the status word
};

// 64 x 64 boxes (x: the contiguous dimension, y: rows, z: matrix of the batch).
struct Maps {
  CUtensorMap a[2], b[2];  // of each segment
  CUtensorMap out[3];
};

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

// What an epilogue works on: a thread is one row of the tile.
struct Tile {
  uint32_t tmem;  // this warp's lanes of the accumulator
  uint8_t* sm;    // staging memory: the tile's operands have been used
  uint32_t sm_addr;
  int row, m0, n0, z;  // row of the tile 0 .. 127, the tile's first output row, column tile's first column, matrix
  int M, N;
};

// The epilogue's four warps meet; epi_all: whether all of them say yes.
__device__ __forceinline__ void epi_sync() { asm volatile("barrier.cta.sync.aligned 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool epi_all(bool ok) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred.aligned q, 1, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)ok)
      : "memory");
  return r != 0;
}

// Eight 16-bit values to columns c .. c + 7 of row r of a staged 64-column box of 128 rows.
__device__ __forceinline__ void stage8(uint8_t* box, int r, int c, const uint4 v) {
  *reinterpret_cast<uint4*>(box + sw128_off(r, c)) = v;
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

// Stores `boxes` staged boxes of 128 rows x 64 columns as columns n0, n0 + 64, ... of rows m0 ... of out (what lies
// outside is left out); by one thread, after the staging threads have met.
__device__ __forceinline__ void store_boxes(const CUtensorMap* out, const Tile& t, uint32_t src, int boxes, int n0) {
  for (int b = 0; b < boxes; ++b)
    for (int y = 0; y < 2; ++y)
      if (n0 + 64 * b < t.N && t.m0 + 64 * y < t.M) tma_store_3d(out, n0 + 64 * b, t.m0 + 64 * y, t.z, src + b * 2 * BOX + y * BOX);
}

// One output tile a CTA, two CTAs on an SM: the one's epilogue runs beside the other's products.
template <typename E, bool A_MN, bool B_MN, bool F16>
__global__ void __launch_bounds__(THREADS, 2) k_gemm(const Args a, const __grid_constant__ Maps maps, const typename E::Args e) {
  extern __shared__ uint8_t dsmem[];
  __shared__ uint64_t full[STAGES], empty[STAGES], acc_full;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_addr(dsmem) + 1023u) & ~1023u;
  volatile int* abort = &abort_flag;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base, TILE);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  pdl_wait();
  pdl_trigger();
  if (a.clear && threadIdx.x == 0 && blockIdx.x + blockIdx.y + blockIdx.z == 0) *a.status = 0;
  const int m0 = blockIdx.y * TILE, n0 = blockIdx.x * E::COLS, z = blockIdx.z;
  const int blocks = a.kb[0] + a.kb[1];
  if (warp == 0) {
    if (lane == 0) {
      int i = 0;
      for (; i < blocks; ++i) {
        const int s = i % STAGES, seg = i >= a.kb[0] ? 1 : 0, k = (seg ? i - a.kb[0] : i) * BK;
        if (i >= STAGES && !wait_ab(&empty[s], ((i / STAGES) - 1) & 1, abort, a.status)) break;
        const uint32_t as = base + s * STAGE, bs = as + 2 * BOX;
        mbar_arrive_expect_tx(&full[s], STAGE);
        for (int h = 0; h < 2; ++h) {
          const int m = m0 + 64 * h, n = E::PAIR ? n0 : n0 + 64 * h;
          const CUtensorMap* bm = E::PAIR ? &maps.b[h] : &maps.b[seg];
          tma_load_3d(as + h * BOX, &maps.a[seg], A_MN ? m : k, A_MN ? k : m, z, &full[s]);
          tma_load_3d(bs + h * BOX, bm, B_MN ? n : k, B_MN ? k : n, z, &full[s]);
        }
      }
      for (int r = (i > STAGES ? i - STAGES : 0); r < i; ++r) mbar_drain(&full[r % STAGES], (r / STAGES) & 1);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f32acc(TILE, TILE, !F16) | (A_MN ? IDESC_A_MN : 0u) | (B_MN ? IDESC_B_MN : 0u);
    int i = 0;
    for (; i < blocks; ++i) {
      const int s = i % STAGES;
      const bool ok = wait_ab(&full[s], (i / STAGES) & 1, abort, a.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t as = base + s * STAGE, bs = as + 2 * BOX;
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks) {
          const uint64_t ad = A_MN ? sw128_desc_mn(as + ks * 2048, BOX) : sw128_desc(as) + (uint64_t)(ks * 2);
          const uint64_t bd = B_MN ? sw128_desc_mn(bs + ks * 2048, BOX) : sw128_desc(bs) + (uint64_t)(ks * 2);
          tc_mma(tmem, ad, bd, idesc, (i > 0 || ks > 0) ? 1u : 0u);
        }
        tc_commit(&empty[s]);
        if (i + 1 == blocks) tc_commit(&acc_full);
      }
      __syncwarp();
    }
    for (int r = (i > STAGES ? i - STAGES : 0); r < i; ++r) mbar_drain(&empty[r % STAGES], (r / STAGES) & 1);
  } else {
    const bool ok = __all_sync(0xffffffffu, wait_ab(&acc_full, 0, abort, a.status));
    if (epi_all(ok)) {  // a warp that gave up takes the others along: they meet again below
      tc_fence_after();
      const int q = warp & 3;
      Tile t;
      t.tmem = tmem + ((uint32_t)(q * 32) << 16);
      t.sm = dsmem + (base - smem_addr(dsmem));
      t.sm_addr = base;
      t.row = q * 32 + lane;
      t.m0 = m0;
      t.n0 = n0;
      t.z = z;
      t.M = a.M;
      t.N = a.N;
      E::run(e, maps, t, warp == 2 && lane == 0);
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, TILE);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
// A batch of matrices [rows][cols] of 16-bit values (rows ld apart, matrices `apart`) in 64 x 64 boxes.
inline bool map_matrix(CUtensorMap* m, const void* p, int64_t cols, int64_t rows, int64_t ld, int64_t batch, int64_t apart) {
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)apart * 2};
  const cuuint32_t box[3] = {64, 64, 1};
  return encode_bf16(m, p, 3, dims, strides, box);
}
inline bool map_matrix(CUtensorMap* m, const void* p, int64_t cols, int64_t rows, int64_t ld) {
  return map_matrix(m, p, cols, rows, ld, 1, ld);  // one matrix: its distance to the next is never used
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

// A launch that may start while the kernel before it drains (each kernel waits for it itself).
template <auto KERNEL, typename... P>
bool launch(dim3 grid, int block, size_t smem, cudaStream_t stream, const P&... args) {
  if (!prepare<KERNEL>(smem)) return false;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, KERNEL, args...) == cudaSuccess;
}

template <typename E, bool A_MN, bool B_MN, bool F16>
bool run(const Args& a, const Maps& m, const typename E::Args& e, int batch, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.N + E::COLS - 1) / E::COLS), (unsigned)((a.M + TILE - 1) / TILE), (unsigned)batch);
  return launch<k_gemm<E, A_MN, B_MN, F16>>(grid, THREADS, SMEM, stream, a, m, e);
}

}  // namespace gemm
}  // namespace flint
