// act8.cu -- activations packed into 8 bits and restored (the format is stated
// in include/dpopt.h): one block of 32 columns is four threads of eight.
#include "ops.cuh"

namespace dpopt {
namespace {

struct Act8Params {
  int64_t rows, cols;
  int64_t groups;  // 8-column groups of one row, rounded up to whole blocks of four
  Mat x;
  Act8Out packed;
  Dbg dbg;
};

constexpr int kActThreads = 256;

template <class T>
__global__ void __launch_bounds__(kActThreads) act8_pack_kernel(const Act8Params p) {
  pdl_enter();
  const int64_t total = p.rows * p.groups;  // a multiple of 4: blocks stay in one warp
  const int64_t stride = (int64_t)gridDim.x * kActThreads;
  const int64_t rounds = (total + stride - 1) / stride;
  int64_t g = (int64_t)blockIdx.x * kActThreads + threadIdx.x;
  for (int64_t it = 0; it < rounds; ++it, g += stride) {
    // threads past the end keep step with their warp on columns past the row's
    const bool live = g < total && dbg_ok(p.dbg, g / p.groups < p.rows);
    const int64_t row = live ? g / p.groups : 0;
    const int64_t col = live ? (g - row * p.groups) * 8 : p.groups * 8;
    float f[8];
    mat_load8<T>(p.x, row, col, p.cols, f);
    act8_store8<T>(p.packed, row, col, p.cols, f);
  }
}

template <class T>
__global__ void __launch_bounds__(kActThreads) act8_unpack_kernel(const Act8Params p) {
  pdl_enter();
  const int64_t total = p.rows * p.groups;
  const int64_t stride = (int64_t)gridDim.x * kActThreads;
  for (int64_t g = (int64_t)blockIdx.x * kActThreads + threadIdx.x; g < total; g += stride) {
    const int64_t row = g / p.groups;
    const int64_t col = (g - row * p.groups) * 8;
    if (!dbg_ok(p.dbg, row < p.rows)) continue;
    float f[8];
    act8_load8(p.packed, row, col, p.cols, f);
    mat_store8<T>(p.x, row, col, p.cols, f);
  }
}

int prepare(Act8Params& p, bool pack, void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx,
            int8_t* codes, int64_t ld_codes, uint8_t* exps, int64_t ld_exps) {
  if (rows < 0 || cols < 0) return fail(DPOPT_ERR_INVALID_ARG, "rows and cols must be >= 0");
  if (!known_dtype(dtype)) return fail(DPOPT_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  Span s[3];
  int n = 0;
  DPOPT_TRY(take_matrix("x", dpopt_matrix{x, ldx}, rows, cols, dtype_size(dtype), !pack, &p.x, s,
                        &n));
  DPOPT_TRY(take_act8("the packed matrix", dpopt_act8{codes, ld_codes, exps, ld_exps}, rows, cols,
                      pack, &p.packed, s, &n));
  DPOPT_TRY(check_overlaps(s, n));
  p.rows = rows;
  p.cols = cols;
  p.groups = (cols + kAct8Block - 1) / kAct8Block * (kAct8Block / 8);
  p.dbg = make_dbg();
  return DPOPT_OK;
}

int run(void (*kern)(const Act8Params), const Act8Params& p, const char* what,
        cudaStream_t stream) {
  if (p.rows == 0 || p.cols == 0) return DPOPT_OK;
  int sms = 0;
  DPOPT_TRY(sm_count(&sms));
  const int64_t blocks = (p.rows * p.groups + kActThreads - 1) / kActThreads;
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)sms * 8);
  return launched(launch_pdl(kern, grid, kActThreads, 0, stream, p), what);
}

}  // namespace
}  // namespace dpopt

using namespace dpopt;

extern "C" {

int dpopt_act8_pack(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                    int8_t* codes, int64_t ld_codes, uint8_t* exps, int64_t ld_exps,
                    dpopt_stream_t stream) {
  Act8Params p;
  DPOPT_TRY(prepare(p, true, const_cast<void*>(x), dtype, rows, cols, ldx, codes, ld_codes, exps,
                    ld_exps));
  auto kern = dtype == DPOPT_GRAD_BF16  ? act8_pack_kernel<bf16>
              : dtype == DPOPT_GRAD_F16 ? act8_pack_kernel<fp16>
                                        : act8_pack_kernel<float>;
  return run(kern, p, "act8 pack", (cudaStream_t)stream);
}

int dpopt_act8_unpack(const int8_t* codes, int64_t ld_codes, const uint8_t* exps, int64_t ld_exps,
                      int64_t rows, int64_t cols, void* x, int dtype, int64_t ldx,
                      dpopt_stream_t stream) {
  Act8Params p;
  DPOPT_TRY(prepare(p, false, x, dtype, rows, cols, ldx, const_cast<int8_t*>(codes), ld_codes,
                    const_cast<uint8_t*>(exps), ld_exps));
  auto kern = dtype == DPOPT_GRAD_BF16  ? act8_unpack_kernel<bf16>
              : dtype == DPOPT_GRAD_F16 ? act8_unpack_kernel<fp16>
                                        : act8_unpack_kernel<float>;
  return run(kern, p, "act8 unpack", (cudaStream_t)stream);
}

}  // extern "C"
