// act8_wgrad.cu -- weight gradient of a linear layer from its packed input:
// dw[i][j] = sum_t dy[t][i] * value(t, j) (+ addend).
//
// Two kernels (three when the tokens are split).  act8_operands_kernel writes the
// packed input's values to scratch in dy's 16-bit type, which holds them exactly,
// and copies dy there too if its rows are not 16-byte aligned.
// act8_wgrad_kernel is a persistent matrix product on the tensor cores: the sum
// runs over tokens, the slow index of both operands, so both are read as they lie
// in memory ("MN-major") and nothing is transposed.
#include <cuda.h>

#include <mutex>

#include "mbar.cuh"
#include "ops.cuh"

namespace dpopt {
namespace {

// ---------------------------------------------------------------------------
// operands
// ---------------------------------------------------------------------------

struct OperandParams {
  int64_t tokens;
  int n, k;
  int64_t x_units, units;  // warp units of 256 columns: the packed input's, and dy's after them
  Act8Out x;
  Mat dy;
  void *x_out, *dy_out;
  int64_t ld_x, ld_dy;  // row strides of the copies, multiples of 8
  Dbg dbg;
};

constexpr int kOperandThreads = 256, kUnit = 256;

template <class T>
__global__ void __launch_bounds__(kOperandThreads)
    act8_operands_kernel(const __grid_constant__ OperandParams p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int xu = (p.k + kUnit - 1) / kUnit, du = (p.n + kUnit - 1) / kUnit;
  const bool vec = p.x.vec && p.k % 8 == 0;
  for (int64_t w = ((int64_t)blockIdx.x * kOperandThreads + threadIdx.x) >> 5; w < p.units;
       w += (int64_t)gridDim.x * (kOperandThreads / 32)) {
    if (w < p.x_units) {
      const int64_t row = w / xu;
      const int c0 = (int)(w - row * xu) * kUnit;
      if (!dbg_ok(p.dbg, row < p.tokens)) continue;
      const int8_t* codes = p.x.codes + row * p.x.ld_codes;
      const uint8_t* exps = p.x.exps + row * p.x.ld_exps;
      T* out = static_cast<T*>(p.x_out) + row * p.ld_x;
      if (vec) {
        const int c = c0 + lane * 8;
        if (c >= p.k) continue;
        float f[8];
        act8_values(*reinterpret_cast<const uint2*>(codes + c), act8_scale(exps[c / kAct8Block]),
                    f);
        *reinterpret_cast<uint4*>(out + c) =
            make_uint4(pack2(f[0], f[1], T()), pack2(f[2], f[3], T()), pack2(f[4], f[5], T()),
                       pack2(f[6], f[7], T()));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = c0 + i * 32 + lane;
          if (c < p.k) out[c] = from_f32<T>((float)codes[c] * act8_scale(exps[c / kAct8Block]));
        }
      }
    } else {
      const int64_t row = (w - p.x_units) / du;
      const int c0 = (int)(w - p.x_units - row * du) * kUnit;
      if (!dbg_ok(p.dbg, row < p.tokens)) continue;
      const T* in = static_cast<const T*>(p.dy.data) + row * p.dy.ld;
      T* out = static_cast<T*>(p.dy_out) + row * p.ld_dy;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + i * 32 + lane;
        if (c < p.n) out[c] = in[c];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------

// A CTA owns a tile of kTileM rows of dw (columns of dy) by BN columns (of the
// input) and steps over kStep tokens at a time.
constexpr int kTileM = 128, kStep = 64;
constexpr int kBoxBytes = 64 * kStep * 2;  // one copied box: 64 columns x kStep tokens
constexpr int kGemmThreads = 192;          // copying warp, issuing warp, four epilogue warps
constexpr int kTileGroup = 16;             // row tiles that run side by side (shared columns in L2)

struct GemmParams {
  int64_t tokens, per_split;  // tokens of a split, a multiple of kStep
  int n, k;
  int tiles_m, tiles_n, splits;
  Mat dw, addend;
  int out_dtype;
  float* partial;  // [split][n][pk] when splits > 1
  int64_t pk;
  long long wait_limit;
  Dbg dbg;
};

template <int BN>
struct GemmShape {
  static constexpr int kBoxes = kTileM / 64 + BN / 64;
  static constexpr int kStageBytes = kBoxes * kBoxBytes;
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr int kSmem = kStages * kStageBytes + 1024;  // 1024-byte aligned
};

// Set when a bounded wait gave up (dpopt_stream_status reads and clears it).
__device__ unsigned int g_gemm_status;

// A wait of at most `limit` cycles; on time-out, or once another role of the CTA
// gave up, false.
__device__ __forceinline__ bool gemm_wait(uint32_t bar, uint32_t parity, long long limit,
                                          volatile int* abort) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_test(bar, parity)) {
    if (*abort) return false;
    if (clock64() - t0 > limit) {
      atomicOr(&g_gemm_status, 1u);
      *abort = 1;
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// Shared-memory matrix descriptor of a 16-bit operand whose 64-element runs along
// the tile's rows (or columns) are 128 bytes, one per token, 128-byte swizzled: the
// next 64 elements start a box further on, the next 8 tokens 1024 bytes further on.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(kBoxBytes >> 4) << 16 |
         (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor: fp32 accumulators, operands of type T, both with the
// token index slow (transposed), a kTileM x BN tile.
template <class T, int BN>
__device__ __forceinline__ constexpr uint32_t instr_desc() {
  constexpr uint32_t fmt = std::is_same_v<T, bf16> ? 1u : 0u;
  return 1u << 4 | fmt << 7 | fmt << 10 | 1u << 15 | 1u << 16 | (uint32_t)(BN / 8) << 17 |
         (uint32_t)(kTileM / 16) << 24;
}

__device__ __forceinline__ void mma_16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Unit u of a launch: the tile's corner and the range of token steps.
struct Unit {
  int m0, n0, split, steps;
  int64_t t0;
};

template <int BN>
__device__ __forceinline__ Unit unit_at(const GemmParams& p, int u) {
  const int tiles = p.tiles_m * p.tiles_n;
  Unit r;
  r.split = u / tiles;
  const int tile = u - r.split * tiles;
  const int group = tile / (kTileGroup * p.tiles_n);
  const int first = group * kTileGroup;
  const int rows = min(kTileGroup, p.tiles_m - first);
  const int local = tile - group * kTileGroup * p.tiles_n;
  r.m0 = (first + local % rows) * kTileM;
  r.n0 = (local / rows) * BN;
  r.t0 = r.split * p.per_split;
  const int64_t t1 = min(p.tokens, r.t0 + p.per_split);
  r.steps = (int)((t1 - r.t0 + kStep - 1) / kStep);
  return r;
}

// 32 columns of one row of a tile: to the partial sums, or with the addend to dw.
template <int BN>
__device__ __forceinline__ void store32(const GemmParams& p, const Unit& u, int row, int col,
                                        const uint32_t (&r)[32]) {
  if (row >= p.n || col >= p.k || !dbg_ok(p.dbg, row >= 0 && col >= 0)) return;
  if (p.splits > 1) {
    float* dst = p.partial + ((int64_t)u.split * p.n + row) * p.pk + col;
#pragma unroll
    for (int i = 0; i < 32; i += 4)
      if (col + i < p.pk)
        *reinterpret_cast<uint4*>(dst + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
    return;
  }
  float f[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]);
  const bool whole = col + 32 <= p.k;
  if (p.addend.data) {
    const int64_t at = row * p.addend.ld + col;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (whole || col + i < p.k) f[i] += ld_any(p.addend.data, p.out_dtype, at + i);
  }
  const int64_t at = row * p.dw.ld + col;
  if (whole && p.dw.vec) {
    if (p.out_dtype == DPOPT_GRAD_F32) {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.dw.data) + at);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        d[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    } else {
      uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dw.data) + at);
      const bool b = p.out_dtype == DPOPT_GRAD_BF16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = b ? pack2(f[8 * i + 2 * j], f[8 * i + 2 * j + 1], bf16())
                   : pack2(f[8 * i + 2 * j], f[8 * i + 2 * j + 1], fp16());
        d[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (col + i < p.k) st_any(p.dw.data, p.out_dtype, at + i, f[i]);
  }
}

// One warp copies boxes into a ring of stages, one issues the products of a stage
// (four of 16 tokens), four bring finished tiles from tensor memory to memory;
// two accumulators let the next tile's products run under a tile's epilogue.
template <class T, int BN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    act8_wgrad_kernel(const __grid_constant__ GemmParams p,
                      const __grid_constant__ CUtensorMap map_a,
                      const __grid_constant__ CUtensorMap map_b) {
  using S = GemmShape<BN>;
  extern __shared__ unsigned char dyn[];
  __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], done[2], taken[2],
      drained;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = (smem_u32(dyn) + 1023u) & ~1023u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&done[a]), 1);
      mbar_init(smem_u32(&taken[a]), 4);
    }
    mbar_init(smem_u32(&drained), 1);
    abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_slot)),
                 "r"(2 * BN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_slot;
  pdl_enter();  // the operands are complete from here on

  const int units = p.tiles_m * p.tiles_n * p.splits;
  if (warp == 0) {
    if (lane == 0) {
      int64_t it = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const Unit q = unit_at<BN>(p, u);
        for (int step = 0; step < q.steps; ++step, ++it) {
          const int s = (int)(it % S::kStages);
          const uint32_t round = (uint32_t)(it / S::kStages);
          if (!(ok = gemm_wait(smem_u32(&empty[s]), (round & 1) ^ 1, p.wait_limit, &abort))) break;
          const uint32_t bar = smem_u32(&full[s]);
          const uint32_t at = ring + s * S::kStageBytes;
          const int y = (int)(q.t0 + (int64_t)step * kStep);
          mbar_arrive_expect_tx(bar, S::kStageBytes);
#pragma unroll
          for (int b = 0; b < kTileM / 64; ++b)
            tma_box(at + b * kBoxBytes, &map_a, q.m0 + b * 64, y, bar);
#pragma unroll
          for (int b = 0; b < BN / 64; ++b)
            tma_box(at + (kTileM / 64 + b) * kBoxBytes, &map_b, q.n0 + b * 64, y, bar);
        }
      }
      // every copy issued lands before this CTA's shared memory goes away
      for (int s = 0; !ok && s < S::kStages; ++s) {
        const int64_t uses = it / S::kStages + (s < it % S::kStages ? 1 : 0);
        const long long t0 = clock64();
        while (uses > 0 && !mbar_test(smem_u32(&full[s]), (uint32_t)((uses - 1) & 1)) &&
               clock64() - t0 < p.wait_limit) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = instr_desc<T, BN>();
      int64_t it = 0;
      int count = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x, ++count) {
        const Unit q = unit_at<BN>(p, u);
        const int a = count & 1;
        if (!(ok = gemm_wait(smem_u32(&taken[a]), ((count >> 1) & 1) ^ 1, p.wait_limit, &abort)))
          break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + a * BN;
        for (int step = 0; step < q.steps; ++step, ++it) {
          const int s = (int)(it % S::kStages);
          const uint32_t round = (uint32_t)(it / S::kStages);
          if (!(ok = gemm_wait(smem_u32(&full[s]), round & 1, p.wait_limit, &abort))) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t at = ring + s * S::kStageBytes;
          const uint64_t da = operand_desc(at);
          const uint64_t db = operand_desc(at + kTileM / 64 * kBoxBytes);
#pragma unroll
          for (int j = 0; j < kStep / 16; ++j)  // 16 tokens are 2048 bytes further on
            mma_16(d, da + j * (2048 >> 4), db + j * (2048 >> 4), idesc, step > 0 || j > 0);
          mma_commit(smem_u32(&empty[s]));
        }
        if (ok) mma_commit(smem_u32(&done[a]));
      }
      if (!ok) {
        // products in flight end before tensor memory is given back
        mma_commit(smem_u32(&drained));
        const long long t0 = clock64();
        while (!mbar_test(smem_u32(&drained), 0) && clock64() - t0 < p.wait_limit) {
        }
      }
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;  // the tensor-memory lanes this warp may read
    int count = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++count) {
      const Unit q = unit_at<BN>(p, u);
      const int a = count & 1;
      const bool ok = gemm_wait(smem_u32(&done[a]), (count >> 1) & 1, p.wait_limit, &abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const int row = q.m0 + quarter * 32 + lane;
      for (int c = 0; c < BN && q.n0 + c < p.k; c += 32) {
        uint32_t r[32];
        tmem_load32(tmem + ((uint32_t)quarter << 21) + a * BN + c, r);
        store32<BN>(p, q, row, q.n0 + c, r);
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&taken[a]));
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN));
}

// dw = the splits' partial sums in order (+ addend); without splits (no tokens)
// the addend, or zeros.
__global__ void __launch_bounds__(256)
    act8_wgrad_sum_kernel(const __grid_constant__ GemmParams p) {
  pdl_enter();
  const int64_t total = (int64_t)p.n * p.k;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total;
       e += (int64_t)gridDim.x * 256) {
    const int64_t i = e / p.k, j = e - i * p.k;
    float s = 0.f;
    for (int q = 0; q < p.splits; ++q) s += p.partial[((int64_t)q * p.n + i) * p.pk + j];
    if (p.addend.data) s += ld_any(p.addend.data, p.out_dtype, i * p.addend.ld + j);
    st_any(p.dw.data, p.out_dtype, i * p.dw.ld + j, s);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

constexpr int64_t kSms = 152, kMinSplit = 256;

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Tile width, and how the tokens are split when there are too few tiles for the
// SMs: functions of the sizes alone.
struct Plan {
  int bn;
  int64_t tiles_m, tiles_n, splits, per_split;
  int64_t ld_x, ld_dy, pk;
  int64_t x_bytes, dy_bytes, partial_bytes;
};

Plan make_plan(int64_t tokens, int64_t n, int64_t k) {
  Plan r{};
  r.tiles_m = (n + kTileM - 1) / kTileM;
  r.bn = r.tiles_m * ((k + 255) / 256) >= kSms ? 256 : 128;
  r.tiles_n = (k + r.bn - 1) / r.bn;
  const int64_t tiles = std::max<int64_t>(1, r.tiles_m * r.tiles_n);
  const int64_t want = std::min(std::max<int64_t>(1, kSms / tiles),
                                std::max<int64_t>(1, (tokens + kMinSplit - 1) / kMinSplit));
  r.per_split = std::max<int64_t>(kStep, up((tokens + want - 1) / want, kStep));
  r.splits = (tokens + r.per_split - 1) / r.per_split;
  r.ld_x = up(k, 64);
  r.ld_dy = up(n, 64);
  r.pk = up(k, 4);
  r.x_bytes = up(tokens * r.ld_x * 2, 256);
  r.dy_bytes = up(tokens * r.ld_dy * 2, 256);
  r.partial_bytes = r.splits > 1 ? r.splits * n * r.pk * 4 : 0;
  return r;
}

// cuTensorMapEncodeTiled, looked up in the driver once.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::once_flag g_encode_once;
EncodeTiled g_encode = nullptr;

int encode(CUtensorMap* map, bool is_bf16, const void* base, int64_t cols, int64_t rows,
           int64_t ld) {
  std::call_once(g_encode_once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<EncodeTiled>(f);
  });
  if (!g_encode) return fail(DPOPT_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, kStep}, step[2] = {1, 1};
  const CUresult e = g_encode(
      map, is_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
      const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (e != CUDA_SUCCESS) return fail(DPOPT_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", (int)e);
  return DPOPT_OK;
}

template <class T, int BN>
int launch_gemm(const GemmParams& p, const CUtensorMap& a, const CUtensorMap& b,
                cudaStream_t stream) {
  auto kern = act8_wgrad_kernel<T, BN>;
  const size_t smem = GemmShape<BN>::kSmem;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return cuda_fail(e, "shared memory size");
  int sms = 0;
  DPOPT_TRY(sm_count(&sms));
  const int64_t units = (int64_t)p.tiles_m * p.tiles_n * p.splits;
  const unsigned grid = (unsigned)std::min<int64_t>(units, sms);
  return launched(launch_pdl(kern, grid, kGemmThreads, smem, stream, p, a, b),
                  "act8 weight gradient");
}

template <class T>
int run_wgrad(const Plan& plan, GemmParams& g, OperandParams& o, unsigned char* scratch,
              cudaStream_t stream) {
  constexpr bool is_bf16 = std::is_same_v<T, bf16>;
  // dy is read in place when its rows are aligned for the copies
  const bool in_place = (uintptr_t)o.dy.data % 16 == 0 && o.dy.ld % 8 == 0;
  o.x_out = scratch;
  o.dy_out = scratch + plan.x_bytes;
  o.ld_x = plan.ld_x;
  o.ld_dy = plan.ld_dy;
  o.x_units = o.tokens * ((o.k + kUnit - 1) / kUnit);
  o.units = o.x_units + (in_place ? 0 : o.tokens * ((o.n + kUnit - 1) / kUnit));
  g.partial = reinterpret_cast<float*>(scratch + plan.x_bytes + plan.dy_bytes);
  int sms = 0;
  DPOPT_TRY(sm_count(&sms));
  CUtensorMap a, b;
  DPOPT_TRY(in_place ? encode(&a, is_bf16, o.dy.data, o.n, o.tokens, o.dy.ld)
                     : encode(&a, is_bf16, o.dy_out, o.n, o.tokens, o.ld_dy));
  DPOPT_TRY(encode(&b, is_bf16, o.x_out, o.k, o.tokens, o.ld_x));
  const unsigned ctas = (unsigned)std::min<int64_t>((o.units + 7) / 8, (int64_t)sms * 8);
  DPOPT_TRY(launched(
      launch_pdl(act8_operands_kernel<T>, ctas, kOperandThreads, 0, stream, o),
      "act8 weight gradient operands"));
  DPOPT_TRY(plan.bn == 256 ? launch_gemm<T, 256>(g, a, b, stream)
                           : launch_gemm<T, 128>(g, a, b, stream));
  return DPOPT_OK;
}

}  // namespace

int take_gemm_status(bool* timed_out) {
  unsigned int st = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&st, g_gemm_status, sizeof st);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyFromSymbol");
  *timed_out = st != 0;
  if (st != 0) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_gemm_status, &zero, sizeof zero);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyToSymbol");
  }
  return DPOPT_OK;
}

}  // namespace dpopt

using namespace dpopt;

extern "C" {

int dpopt_act8_wgrad_scratch_bytes(int64_t tokens, int64_t n, int64_t k, int64_t* bytes_out) {
  if (!bytes_out || tokens < 0 || n < 0 || k < 0)
    return fail(DPOPT_ERR_INVALID_ARG, "wgrad scratch: null output or a negative size");
  const int64_t limit = (int64_t)1 << 31;
  if (tokens >= limit || n >= limit || k >= limit)
    return fail(DPOPT_ERR_UNSUPPORTED, "sizes must be below 2^31");
  const Plan plan = make_plan(tokens, n, k);
  *bytes_out = plan.x_bytes + plan.dy_bytes + plan.partial_bytes;
  return DPOPT_OK;
}

int dpopt_act8_wgrad(const void* dy, int dtype, int64_t ld_dy, const int8_t* codes,
                     int64_t ld_codes, const uint8_t* exps, int64_t ld_exps, int64_t tokens,
                     int64_t n, int64_t k, void* dw, int out_dtype, int64_t ld_dw,
                     const void* addend, int64_t ld_addend, void* scratch, int64_t scratch_bytes,
                     dpopt_stream_t stream) {
  if (tokens < 0 || n < 0 || k < 0)
    return fail(DPOPT_ERR_INVALID_ARG, "tokens, n and k must be >= 0");
  if (!known_dtype(dtype)) return fail(DPOPT_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (!known_dtype(out_dtype))
    return fail(DPOPT_ERR_INVALID_ARG, "unknown out_dtype %d", out_dtype);
  if (dtype == DPOPT_GRAD_F32)
    return fail(DPOPT_ERR_UNSUPPORTED, "dy must be bf16 or fp16");
  int64_t need = 0;
  DPOPT_TRY(dpopt_act8_wgrad_scratch_bytes(tokens, n, k, &need));
  if (n == 0 || k == 0) return DPOPT_OK;
  GemmParams g{};
  OperandParams o{};
  Span s[8];
  int cnt = 0;
  Mat dummy;
  const int64_t es = dtype_size(dtype), os = dtype_size(out_dtype);
  DPOPT_TRY(take_matrix("dw", dpopt_matrix{dw, ld_dw}, n, k, os, true, &g.dw, s, &cnt));
  if (addend) {
    DPOPT_TRY(take_matrix("addend", dpopt_matrix{const_cast<void*>(addend), ld_addend}, n, k, os,
                          false, &g.addend, s, &cnt));
    if (addend == dw && (n == 1 || ld_addend == ld_dw)) s[1].hi = s[1].lo;  // in place
  }
  DPOPT_TRY(take_matrix("dy", dpopt_matrix{const_cast<void*>(dy), ld_dy}, tokens, n, es, false,
                        &o.dy, s, &cnt));
  DPOPT_TRY(take_act8("the packed input",
                      dpopt_act8{const_cast<int8_t*>(codes), ld_codes,
                                 const_cast<uint8_t*>(exps), ld_exps},
                      tokens, k, false, &o.x, s, &cnt));
  if (need > 0) {
    if (!scratch || (uintptr_t)scratch % 256)
      return fail(DPOPT_ERR_INVALID_ARG, "scratch must be non-null and 256-byte aligned");
    if (scratch_bytes < need)
      return fail(DPOPT_ERR_INVALID_ARG, "scratch holds %lld bytes, %lld are needed",
                  (long long)scratch_bytes, (long long)need);
    DPOPT_TRY(
        take_matrix("scratch", dpopt_matrix{scratch, need}, 1, need, 1, true, &dummy, s, &cnt));
  }
  DPOPT_TRY(check_overlaps(s, cnt));
  const Plan plan = make_plan(tokens, n, k);
  if (plan.tiles_m * plan.tiles_n * std::max<int64_t>(1, plan.splits) > INT32_MAX / 2)
    return fail(DPOPT_ERR_UNSUPPORTED, "too many tiles");
  o.tokens = g.tokens = tokens;
  o.n = g.n = (int)n;
  o.k = g.k = (int)k;
  o.dbg = g.dbg = make_dbg();
  g.per_split = plan.per_split;
  g.tiles_m = (int)plan.tiles_m;
  g.tiles_n = (int)plan.tiles_n;
  g.splits = (int)plan.splits;
  g.pk = plan.pk;
  g.out_dtype = out_dtype;
  g.wait_limit = kWaitLimitCycles;
  const cudaStream_t st = (cudaStream_t)stream;
  if (tokens > 0) {
    unsigned char* at = static_cast<unsigned char*>(scratch);
    DPOPT_TRY(dtype == DPOPT_GRAD_BF16 ? run_wgrad<bf16>(plan, g, o, at, st)
                                       : run_wgrad<fp16>(plan, g, o, at, st));
    if (plan.splits == 1) return DPOPT_OK;
  }
  int sms = 0;
  DPOPT_TRY(sm_count(&sms));
  const unsigned ctas = (unsigned)std::min<int64_t>((n * k + 255) / 256, (int64_t)sms * 8);
  return launched(launch_pdl(act8_wgrad_sum_kernel, ctas, 256, 0, st, g),
                  "act8 weight gradient sum");
}

}  // extern "C"
