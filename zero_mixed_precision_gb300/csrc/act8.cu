// act8.cu -- activations packed into 8 bits and restored (the format is stated
// in include/dpopt.h).
//
// Both directions move 3.03 bytes per 16-bit element and are bound by memory,
// the packing nearly as much by arithmetic (two thirds of the issue slots: the
// largest magnitude, one fused multiply-add per two codes that scales and rounds,
// byte permutes).  A warp takes 256 columns of a row, the next unit's loads in
// flight while it works on one.  8192 x 8192 bf16: 36.7 us packing, 35.8 us restoring,
// 5.5 and 5.7 TB/s (82 and 84 % of the measured copy rate); fp32 55 and 64 us, 6.2
// and 5.2 TB/s (the restoring writes four bytes for each that it reads).
// Rows that are not 16-byte aligned are read and written by whole aligned chunks all
// the same, shifted between lanes (8192 x 8191: 65 and 61 us; element by element, a
// warp's lanes on neighbouring columns, they were 103 and 90).
#include "ops.cuh"

namespace dpopt {
namespace {

struct Act8Params {
  int64_t rows;
  int cols;
  UnitSteps steps;
  Mat x;
  Act8Out packed;
  Dbg dbg;
};

constexpr int kActThreads = 256;

template <class T, bool VEC>
__global__ void __launch_bounds__(kActThreads)
    act8_pack_kernel(const __grid_constant__ Act8Params p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  UnitWalk at(p.steps, kActThreads);
  UnitFrag<T, VEC> ahead;
  if (at.row < p.rows) ahead.load(p.x, p.rows, at.row, lane, p.cols, at.unit * kUnitCols);
  while (at.row < p.rows && dbg_ok(p.dbg, at.unit < p.steps.units)) {
    const int64_t row = at.row;
    const int c0 = at.unit * kUnitCols;
    float f[8];
    ahead.widen(f, c0 + lane * 8, p.cols);
    at.next(p.steps);
    if (at.row < p.rows) ahead.load(p.x, p.rows, at.row, lane, p.cols, at.unit * kUnitCols);
    unit_pack<T, VEC>(p.packed, row, lane, p.cols, c0, f);
  }
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kActThreads)
    act8_unpack_kernel(const __grid_constant__ Act8Params p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  UnitWalk at(p.steps, kActThreads);
  CodeFrag<VEC> ahead;
  if (at.row < p.rows) ahead.load(p.packed, p.rows, at.row, lane, p.cols, at.unit * kUnitCols);
  while (at.row < p.rows && dbg_ok(p.dbg, at.unit < p.steps.units)) {
    const int64_t row = at.row;
    const int c0 = at.unit * kUnitCols;
    float f[8];
    ahead.values(f);
    at.next(p.steps);
    if (at.row < p.rows) ahead.load(p.packed, p.rows, at.row, lane, p.cols, at.unit * kUnitCols);
    unit_store<T, VEC>(p.x, row, lane, p.cols, c0, f);
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
  if (cols > INT32_MAX - kUnitCols) return fail(DPOPT_ERR_UNSUPPORTED, "cols must be below 2^31");
  p.rows = rows;
  p.cols = (int)cols;
  p.dbg = make_dbg();
  return DPOPT_OK;
}

using Kernel = void (*)(const Act8Params);

int run(Kernel vec, Kernel elem, Act8Params& p, const char* what, cudaStream_t stream) {
  if (p.rows == 0 || p.cols == 0) return DPOPT_OK;
  int sms = 0;
  DPOPT_TRY(sm_count(&sms));
  const unsigned grid = unit_grid(p.rows, p.cols, sms * 8, kActThreads, &p.steps);
  const bool v = p.cols % 8 == 0 && p.x.vec && p.packed.vec;
  return launched(launch_pdl(v ? vec : elem, grid, kActThreads, 0, stream, p), what);
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
  const cudaStream_t st = (cudaStream_t)stream;
  if (dtype == DPOPT_GRAD_BF16)
    return run(act8_pack_kernel<bf16, true>, act8_pack_kernel<bf16, false>, p, "act8 pack", st);
  if (dtype == DPOPT_GRAD_F16)
    return run(act8_pack_kernel<fp16, true>, act8_pack_kernel<fp16, false>, p, "act8 pack", st);
  return run(act8_pack_kernel<float, true>, act8_pack_kernel<float, false>, p, "act8 pack", st);
}

int dpopt_act8_unpack(const int8_t* codes, int64_t ld_codes, const uint8_t* exps, int64_t ld_exps,
                      int64_t rows, int64_t cols, void* x, int dtype, int64_t ldx,
                      dpopt_stream_t stream) {
  Act8Params p;
  DPOPT_TRY(prepare(p, false, x, dtype, rows, cols, ldx, const_cast<int8_t*>(codes), ld_codes,
                    const_cast<uint8_t*>(exps), ld_exps));
  const cudaStream_t st = (cudaStream_t)stream;
  if (dtype == DPOPT_GRAD_BF16)
    return run(act8_unpack_kernel<bf16, true>, act8_unpack_kernel<bf16, false>, p, "act8 unpack", st);
  if (dtype == DPOPT_GRAD_F16)
    return run(act8_unpack_kernel<fp16, true>, act8_unpack_kernel<fp16, false>, p, "act8 unpack", st);
  return run(act8_unpack_kernel<float, true>, act8_unpack_kernel<float, false>, p, "act8 unpack", st);
}

}  // extern "C"
