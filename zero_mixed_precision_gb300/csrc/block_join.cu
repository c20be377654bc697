// block_join.cu -- the join between two transformer blocks (the norm after the
// block, gate, residual scale, the norm before the next block) and its
// gradient; the formulas stand in include/dpopt.h.
#include <cmath>

#include "ops.cuh"

namespace dpopt {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

struct JoinParams {
  int64_t rows, cols;
  int64_t groups;  // 8-column groups of a row, rounded up to whole 32-column blocks
  int param_dtype;
  float eps, res_scale, branch_scale;
  int64_t gate_rows;
  Mat h, y, gate, h_out, u;
  const void *w_post, *w_pre;
  float *rstd_post, *rstd_pre;
  Act8Out y8, h8, u8;
  Dbg dbg;
};

// Sum over the CTA of N values at once, the same bits in every thread: each
// warp's butterfly, then the warps' sums in warp order.
template <int N>
__device__ __forceinline__ void cta_sum(float (&x)[N], float (*slot)[N]) {
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = warp_sum(x[i]);
  __syncthreads();  // the slots' earlier readers are done
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) slot[warp][i] = x[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) x[i] += slot[w][i];
  }
}

// Eight values of a weight, or ones.
__device__ __forceinline__ void weight8(const void* w, int dtype, int64_t col, int64_t cols,
                                        float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = w && col + i < cols ? ld_any(w, dtype, col + i) : 1.f;
}

template <class T>
__device__ __forceinline__ void round8(const float (&f)[8], float (&r)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = to_f32(from_f32<T>(f[i]));
}

__device__ __forceinline__ int64_t gate_row_of(int64_t gate_rows, int64_t row) {
  return gate_rows > 0 ? row / gate_rows : 0;
}

// One CTA per row, the fp32 row of h_out in shared memory between the two
// norms: any width, stride and alignment.
template <class T>
__global__ void __launch_bounds__(kJoinThreads) block_join_kernel(const JoinParams p) {
  pdl_enter();
  extern __shared__ float hrow[];  // groups * 8
  __shared__ float slot[kJoinWarps][1];
  const int64_t rounds = (p.groups + kJoinThreads - 1) / kJoinThreads;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    float rpost = 1.f;
    if (p.rstd_post) {
      float ss[1] = {0.f};
      for (int64_t g = threadIdx.x; g < p.groups; g += kJoinThreads) {
        float y[8];
        mat_load8<T>(p.y, row, g * 8, p.cols, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(y[i], y[i], ss[0]);
      }
      cta_sum<1>(ss, slot);
      rpost = 1.f / sqrtf(ss[0] / (float)p.cols + p.eps);
      if (threadIdx.x == 0) p.rstd_post[row] = rpost;
    }
    const int64_t grow = gate_row_of(p.gate_rows, row);
    float ss[1] = {0.f};
    for (int64_t it = 0; it < rounds; ++it) {
      const int64_t g = it * kJoinThreads + threadIdx.x;
      const int64_t col = g * 8;  // may lie past the row: zeros, nothing stored
      float y[8], h[8], w[8], hr[8];
      mat_load8<T>(p.y, row, col, p.cols, y);
      mat_load8<T>(p.h, row, col, p.cols, h);
      weight8(p.w_post, p.param_dtype, col, p.cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float gate = p.gate.data && col + i < p.cols
                               ? ld_any(p.gate.data, p.param_dtype, grow * p.gate.ld + col + i)
                               : 1.f;
        const float z = y[i] * rpost * w[i];
        h[i] = p.res_scale * h[i] + p.branch_scale * gate * z;
        if (col + i < p.cols) ss[0] = fmaf(h[i], h[i], ss[0]);
      }
      mat_store8<T>(p.h_out, row, col, p.cols, h);
      if (p.y8.codes) act8_store8<T>(p.y8, row, col, p.cols, y);
      if (p.h8.codes) {
        round8<T>(h, hr);
        act8_store8<T>(p.h8, row, col, p.cols, hr);
      }
      if (g < p.groups) {
#pragma unroll
        for (int i = 0; i < 8; ++i) hrow[col + i] = h[i];
      }
    }
    if (!p.u.data) continue;
    cta_sum<1>(ss, slot);
    const float rpre = 1.f / sqrtf(ss[0] / (float)p.cols + p.eps);
    if (threadIdx.x == 0) p.rstd_pre[row] = rpre;
    for (int64_t it = 0; it < rounds; ++it) {
      const int64_t g = it * kJoinThreads + threadIdx.x;
      const int64_t col = g * 8;
      float u[8], w[8], ur[8];
      weight8(p.w_pre, p.param_dtype, col, p.cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = col + i < p.cols ? hrow[col + i] * rpre * w[i] : 0.f;
      mat_store8<T>(p.u, row, col, p.cols, u);
      if (p.u8.codes) {
        round8<T>(u, ur);
        act8_store8<T>(p.u8, row, col, p.cols, ur);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------

// Sums over rows: the rows are cut into at most kJoinParts runs, whose number
// and borders depend on the row count alone.  Each run's CTA leaves one partial
// row per sum in scratch and the finish kernel adds them in order, so the
// result does not depend on the GPU or on timing.
constexpr int kJoinParts = 304;

__host__ __device__ inline int64_t part_rows(int64_t rows) {
  const int64_t parts = rows < kJoinParts ? rows : kJoinParts;
  return parts == 0 ? 1 : (rows + parts - 1) / parts;
}
__host__ __device__ inline int64_t part_count(int64_t rows) {
  return (rows + part_rows(rows) - 1) / part_rows(rows);
}

// Partial rows of one part: dw_pre, dw_post, and up to two of dgate (of the
// part's first gate row, and of its last when that is another one; gate rows
// that lie inside a part are stored at once).
enum { kPartWPre = 0, kPartWPost = 1, kPartGateFirst = 2, kPartGateLast = 3, kPartSlots = 4 };

struct JoinGradParams {
  int64_t rows, cols, groups;
  int param_dtype;
  float res_scale, branch_scale;
  int64_t gate_rows;
  Mat dh_out, du, y, h_out, gate, dh, dy, dgate;
  Act8Out y8, h8;
  const void *w_post, *w_pre;
  const float *rstd_post, *rstd_pre;
  void *dw_post, *dw_pre;
  float* partial;  // [part][kPartSlots][groups * 8]
  Dbg dbg;
};

__device__ __forceinline__ float* part_row(const JoinGradParams& p, int64_t part, int slot) {
  return p.partial + (part * kPartSlots + slot) * p.groups * 8;
}

// Rows [lo, hi) that use the gate row of `row`.
__host__ __device__ inline void gate_span(int64_t gate_rows, int64_t rows, int64_t row, int64_t* lo,
                                          int64_t* hi) {
  *lo = gate_rows > 0 ? row / gate_rows * gate_rows : 0;
  *hi = gate_rows > 0 && *lo + gate_rows < rows ? *lo + gate_rows : rows;
}

// One CTA per run of rows.  Per row one pass forms three sums,
//   s = <w_pre du, h>,  a = <q, dh_out + r1 w_pre du>,  b = <q, h>,
//   q = w_post gate y,
// from which <w_post dz, y> = branch (a - r1^3 s / C b); a second pass forms the
// outputs.  The sums over rows stay in shared memory, each column owned by one
// thread.
template <class T>
__global__ void __launch_bounds__(kJoinThreads) block_join_grad_kernel(const JoinGradParams p) {
  pdl_enter();
  extern __shared__ float acc[];  // [3][groups * 8]: dw_pre, dw_post, dgate
  __shared__ float slot[kJoinWarps][3];
  const int64_t width = p.groups * 8;
  const int64_t part = blockIdx.x;
  const int64_t lo = part * part_rows(p.rows);
  const int64_t hi = min(p.rows, lo + part_rows(p.rows));
  const float inv_c = 1.f / (float)p.cols;
  for (int64_t g = threadIdx.x; g < p.groups; g += kJoinThreads)
    for (int i = 0; i < 24; ++i) acc[(i >> 3) * width + g * 8 + (i & 7)] = 0.f;
  bool first_gate = true;
  for (int64_t row = lo; row < hi; ++row) {
    const int64_t grow = gate_row_of(p.gate_rows, row);
    const float r1 = p.du.data ? p.rstd_pre[row] : 0.f;
    const float r2 = p.rstd_post ? p.rstd_post[row] : 1.f;
    auto load = [&](int64_t col, float (&d)[8], float (&t)[8], float (&h)[8], float (&y)[8],
                    float (&wp)[8], float (&g)[8]) {
      mat_load8<T>(p.dh_out, row, col, p.cols, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = h[i] = 0.f;
      if (p.du.data) {
        mat_load8<T>(p.du, row, col, p.cols, t);
        if (p.h8.codes)
          act8_load8(p.h8, row, col, p.cols, h);
        else
          mat_load8<T>(p.h_out, row, col, p.cols, h);
      }
      if (p.y8.codes)
        act8_load8(p.y8, row, col, p.cols, y);
      else
        mat_load8<T>(p.y, row, col, p.cols, y);
      weight8(p.w_post, p.param_dtype, col, p.cols, wp);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        g[i] = p.gate.data && col + i < p.cols
                   ? ld_any(p.gate.data, p.param_dtype, grow * p.gate.ld + col + i)
                   : 1.f;
    };
    float sum[3] = {0.f, 0.f, 0.f};
    for (int64_t gi = threadIdx.x; gi < p.groups; gi += kJoinThreads) {
      const int64_t col = gi * 8;
      float d[8], t[8], h[8], y[8], wp[8], g[8], w[8];
      load(col, d, t, h, y, wp, g);
      weight8(p.w_pre, p.param_dtype, col, p.cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (col + i >= p.cols) continue;
        const float q = wp[i] * g[i] * y[i], wd = w[i] * t[i];
        sum[0] = fmaf(wd, h[i], sum[0]);
        sum[1] = fmaf(q, fmaf(r1, wd, d[i]), sum[1]);
        sum[2] = fmaf(q, h[i], sum[2]);
      }
    }
    cta_sum<3>(sum, slot);
    const float k1 = r1 * r1 * r1 * sum[0] * inv_c;
    const float k2 = p.rstd_post
                         ? r2 * r2 * r2 * p.branch_scale * (sum[1] - k1 * sum[2]) * inv_c
                         : 0.f;
    for (int64_t gi = threadIdx.x; gi < p.groups; gi += kJoinThreads) {
      const int64_t col = gi * 8;
      float d[8], t[8], h[8], y[8], wp[8], g[8], w[8];
      load(col, d, t, h, y, wp, g);
      weight8(p.w_pre, p.param_dtype, col, p.cols, w);
      float dh[8], dy[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float full = fmaf(r1, w[i] * t[i], d[i]) - k1 * h[i];
        const float dz = p.branch_scale * g[i] * full;
        dh[i] = p.res_scale * full;
        dy[i] = p.rstd_post ? r2 * wp[i] * dz - k2 * y[i] : dz;
        acc[col + i] = fmaf(t[i], h[i] * r1, acc[col + i]);
        acc[width + col + i] = fmaf(dz, y[i] * r2, acc[width + col + i]);
        acc[2 * width + col + i] =
            fmaf(p.branch_scale * full, y[i] * r2 * wp[i], acc[2 * width + col + i]);
      }
      if (p.dh.data) mat_store8<T>(p.dh, row, col, p.cols, dh);
      mat_store8<T>(p.dy, row, col, p.cols, dy);
    }
    if (p.dgate.data) {
      int64_t glo, ghi;
      gate_span(p.gate_rows, p.rows, row, &glo, &ghi);
      if (row + 1 == hi || row + 1 == ghi) {  // the last row here of its gate row
        const bool inside = glo >= lo && ghi <= hi;
        float* out = part_row(p, part, first_gate ? kPartGateFirst : kPartGateLast);
        for (int64_t gi = threadIdx.x; gi < p.groups; gi += kJoinThreads)
          for (int64_t col = gi * 8; col < gi * 8 + 8; ++col) {
            if (col >= p.cols) continue;
            const float x = acc[2 * width + col];
            if (inside)
              st_any(p.dgate.data, p.param_dtype, grow * p.dgate.ld + col, x);
            else
              out[col] = x;
            acc[2 * width + col] = 0.f;
          }
        first_gate = false;
      }
    }
  }
  for (int64_t gi = threadIdx.x; gi < p.groups; gi += kJoinThreads)
    for (int64_t col = gi * 8; col < gi * 8 + 8; ++col) {
      if (p.dw_pre) part_row(p, part, kPartWPre)[col] = acc[col];
      if (p.dw_post) part_row(p, part, kPartWPost)[col] = acc[width + col];
    }
}

// Adds the parts' partial rows.  blockIdx.y: 0 dw_pre, 1 dw_post, 2 + q the gate
// row that begins in part q and reaches into part q + 1 (with one gate row
// for all rows, q = 0).  32 columns x 8 runs of parts per CTA; the runs' sums
// are added in order.
constexpr int kFinishRuns = 8;

__global__ void __launch_bounds__(32 * kFinishRuns)
block_join_finish_kernel(const JoinGradParams p) {
  pdl_enter();
  __shared__ float run_sum[kFinishRuns][33];
  const int64_t parts = part_count(p.rows), per = part_rows(p.rows);
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  int slot = blockIdx.y;
  int64_t first = 0, last = parts;  // parts [first, last)
  int64_t out_row = 0;
  void* out = blockIdx.y == 0 ? p.dw_pre : p.dw_post;
  if (blockIdx.y >= 2) {
    out = p.dgate.data;
    const int64_t q = blockIdx.y - 2;
    if (p.rows > 0) {
      int64_t glo, ghi;
      const int64_t end = min(p.rows, (q + 1) * per);
      gate_span(p.gate_rows, p.rows, end - 1, &glo, &ghi);
      if (glo < q * per || (ghi <= end && !(q == 0 && parts == 0))) out = nullptr;
      first = q;
      last = (ghi + per - 1) / per;
      out_row = gate_row_of(p.gate_rows, end - 1);
    }
  }
  if (!out) return;
  float s = 0.f;
  const int64_t each = (last - first + kFinishRuns - 1) / kFinishRuns;
  const int64_t a = first + run * each, b = min(last, a + each);
  if (col < p.cols) {
    for (int64_t q = a; q < b; ++q) {
      int use = slot;
      if (blockIdx.y >= 2) {
        int64_t glo, ghi;
        gate_span(p.gate_rows, p.rows, q * per, &glo, &ghi);
        use = gate_row_of(p.gate_rows, q * per) == out_row ? kPartGateFirst : kPartGateLast;
      }
      s += part_row(p, q, use)[col];
    }
  }
  run_sum[run][lane] = s;
  __syncthreads();
  if (run != 0 || col >= p.cols) return;
  for (int i = 1; i < kFinishRuns; ++i) s += run_sum[i][lane];
  if (blockIdx.y < 2)
    st_any(out, p.param_dtype, col, s);
  else
    st_any(out, p.param_dtype, out_row * p.dgate.ld + col, s);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

int check_common(int64_t rows, int64_t cols, int dtype, int param_dtype, int64_t gate_rows,
                 float res_scale, float branch_scale) {
  if (rows < 0 || cols < 0) return fail(DPOPT_ERR_INVALID_ARG, "rows and cols must be >= 0");
  if (cols > DPOPT_JOIN_MAX_COLS)
    return fail(DPOPT_ERR_UNSUPPORTED, "cols %lld exceeds %d", (long long)cols,
                DPOPT_JOIN_MAX_COLS);
  if (!known_dtype(dtype)) return fail(DPOPT_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (!known_dtype(param_dtype))
    return fail(DPOPT_ERR_INVALID_ARG, "unknown param_dtype %d", param_dtype);
  if (gate_rows < 0) return fail(DPOPT_ERR_INVALID_ARG, "gate_rows must be >= 0");
  if (!std::isfinite(res_scale) || !std::isfinite(branch_scale))
    return fail(DPOPT_ERR_INVALID_ARG, "res_scale and branch_scale must be finite");
  return DPOPT_OK;
}

int64_t gate_count(int64_t rows, int64_t gate_rows) {
  return gate_rows == 0 ? 1 : (rows + gate_rows - 1) / gate_rows;
}

bool same(const dpopt_matrix& a, const dpopt_matrix& b, int64_t rows) {
  return a.data == b.data && (rows <= 1 || a.ld == b.ld);
}

int64_t round_groups(int64_t cols) {
  return (cols + kAct8Block - 1) / kAct8Block * (kAct8Block / 8);
}

template <class K>
int allow_smem(K kern, size_t bytes) {
  if (bytes <= 40 * 1024) return DPOPT_OK;  // 48 KB without asking, static arrays included
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  return e == cudaSuccess ? DPOPT_OK : cuda_fail(e, "shared memory size");
}

}  // namespace
}  // namespace dpopt

using namespace dpopt;

extern "C" {

int dpopt_block_join(const dpopt_block_join_args* a, dpopt_stream_t stream) {
  if (!a) return fail(DPOPT_ERR_INVALID_ARG, "args is null");
  DPOPT_TRY(check_common(a->rows, a->cols, a->dtype, a->param_dtype, a->gate_rows, a->res_scale,
                         a->branch_scale));
  if (!std::isfinite(a->eps) || a->eps < 0.f)
    return fail(DPOPT_ERR_INVALID_ARG, "eps must be finite, >= 0");
  if (a->rows == 0 || a->cols == 0) return DPOPT_OK;
  if (a->w_post && !a->rstd_post)
    return fail(DPOPT_ERR_INVALID_ARG, "w_post without rstd_post (no norm after the block)");
  if (!a->u.data && (a->w_pre || a->rstd_pre || a->u8.codes))
    return fail(DPOPT_ERR_INVALID_ARG, "w_pre, rstd_pre or u8 without u");
  if (a->u.data && !a->rstd_pre) return fail(DPOPT_ERR_INVALID_ARG, "rstd_pre is null");
  const int64_t rows = a->rows, cols = a->cols, es = dtype_size(a->dtype);
  const int64_t ps = dtype_size(a->param_dtype);
  JoinParams p{};
  Span s[24];
  int n = 0;
  DPOPT_TRY(take_matrix("h", a->h, rows, cols, es, false, &p.h, s, &n));
  DPOPT_TRY(take_matrix("h_out", a->h_out, rows, cols, es, true, &p.h_out, s, &n));
  if (same(a->h, a->h_out, rows)) s[0].hi = s[0].lo;  // in place
  DPOPT_TRY(take_matrix("y", a->y, rows, cols, es, false, &p.y, s, &n));
  if (a->u.data) DPOPT_TRY(take_matrix("u", a->u, rows, cols, es, true, &p.u, s, &n));
  Mat dummy;
  if (a->gate.data)
    DPOPT_TRY(take_matrix("gate", a->gate, gate_count(rows, a->gate_rows), cols, ps, false,
                          &p.gate, s, &n));
  auto vec = [&](const char* name, const void* q, int64_t len, int64_t size, bool w) {
    return q ? take_matrix(name, dpopt_matrix{const_cast<void*>(q), len}, 1, len, size, w, &dummy,
                           s, &n)
             : DPOPT_OK;
  };
  DPOPT_TRY(vec("w_post", a->w_post, cols, ps, false));
  DPOPT_TRY(vec("w_pre", a->w_pre, cols, ps, false));
  DPOPT_TRY(vec("rstd_post", a->rstd_post, rows, 4, true));
  DPOPT_TRY(vec("rstd_pre", a->rstd_pre, rows, 4, true));
  if (a->y8.codes) DPOPT_TRY(take_act8("y8", a->y8, rows, cols, true, &p.y8, s, &n));
  if (a->h8.codes) DPOPT_TRY(take_act8("h8", a->h8, rows, cols, true, &p.h8, s, &n));
  if (a->u8.codes) DPOPT_TRY(take_act8("u8", a->u8, rows, cols, true, &p.u8, s, &n));
  DPOPT_TRY(check_overlaps(s, n));
  p.rows = rows;
  p.cols = cols;
  p.groups = round_groups(cols);
  p.param_dtype = a->param_dtype;
  p.eps = a->eps;
  p.res_scale = a->res_scale;
  p.branch_scale = a->branch_scale;
  p.gate_rows = a->gate_rows;
  p.w_post = a->w_post;
  p.w_pre = a->w_pre;
  p.rstd_post = a->rstd_post;
  p.rstd_pre = a->rstd_pre;
  p.dbg = make_dbg();
  int sms = 0;
  DPOPT_TRY(sm_count(&sms));
  auto kern = a->dtype == DPOPT_GRAD_BF16  ? block_join_kernel<bf16>
              : a->dtype == DPOPT_GRAD_F16 ? block_join_kernel<fp16>
                                           : block_join_kernel<float>;
  const size_t smem = (size_t)p.groups * 8 * sizeof(float);
  DPOPT_TRY(allow_smem(kern, smem));
  const unsigned grid = (unsigned)std::min<int64_t>(rows, (int64_t)sms * 8);
  return launched(launch_pdl(kern, grid, kJoinThreads, smem, (cudaStream_t)stream, p),
                  "block join");
}

int dpopt_block_join_scratch_bytes(int64_t rows, int64_t cols, int64_t gate_rows,
                                   int64_t* bytes_out) {
  if (!bytes_out || rows < 0 || cols < 0 || gate_rows < 0)
    return fail(DPOPT_ERR_INVALID_ARG, "block join scratch: null output or a negative size");
  if (cols > DPOPT_JOIN_MAX_COLS)
    return fail(DPOPT_ERR_UNSUPPORTED, "cols %lld exceeds %d", (long long)cols,
                DPOPT_JOIN_MAX_COLS);
  *bytes_out = part_count(rows) * kPartSlots * round_groups(cols) * 8 * (int64_t)sizeof(float);
  return DPOPT_OK;
}

int dpopt_block_join_backward(const dpopt_block_join_grad_args* a, dpopt_stream_t stream) {
  if (!a) return fail(DPOPT_ERR_INVALID_ARG, "args is null");
  DPOPT_TRY(check_common(a->rows, a->cols, a->dtype, a->param_dtype, a->gate_rows, a->res_scale,
                         a->branch_scale));
  // without rows there is nothing to read: only the sums are written, as zeros
  const bool some = a->rows > 0 && a->cols > 0;
  const bool pre = a->du.data != nullptr;
  if (some) {
    if ((a->y.data != nullptr) == (a->y8.codes != nullptr))
      return fail(DPOPT_ERR_INVALID_ARG, "exactly one of y and y8 must be given");
    if (pre && (a->h_out.data != nullptr) == (a->h8.codes != nullptr))
      return fail(DPOPT_ERR_INVALID_ARG, "exactly one of h_out and h8 must be given with du");
    if (!pre && (a->h_out.data || a->h8.codes || a->w_pre || a->rstd_pre || a->dw_pre))
      return fail(DPOPT_ERR_INVALID_ARG, "h_out, h8, w_pre, rstd_pre or dw_pre without du");
    if (pre && !a->rstd_pre) return fail(DPOPT_ERR_INVALID_ARG, "rstd_pre is null");
    if ((a->w_post || a->dw_post) && !a->rstd_post)
      return fail(DPOPT_ERR_INVALID_ARG, "w_post or dw_post without rstd_post");
  }
  if (a->dgate.data && !a->gate.data) return fail(DPOPT_ERR_INVALID_ARG, "dgate without gate");
  if (a->cols == 0) return DPOPT_OK;
  const int64_t rows = a->rows, cols = a->cols, es = dtype_size(a->dtype);
  const int64_t ps = dtype_size(a->param_dtype);
  JoinGradParams p{};
  Span s[24];
  int n = 0;
  DPOPT_TRY(take_matrix("dh_out", a->dh_out, rows, cols, es, false, &p.dh_out, s, &n));
  if (a->dh.data) {
    DPOPT_TRY(take_matrix("dh", a->dh, rows, cols, es, true, &p.dh, s, &n));
    if (same(a->dh, a->dh_out, rows)) s[0].hi = s[0].lo;  // in place
  }
  DPOPT_TRY(take_matrix("dy", a->dy, rows, cols, es, true, &p.dy, s, &n));
  if (pre) DPOPT_TRY(take_matrix("du", a->du, rows, cols, es, false, &p.du, s, &n));
  if (a->y.data) DPOPT_TRY(take_matrix("y", a->y, rows, cols, es, false, &p.y, s, &n));
  if (a->h_out.data)
    DPOPT_TRY(take_matrix("h_out", a->h_out, rows, cols, es, false, &p.h_out, s, &n));
  if (a->y8.codes) DPOPT_TRY(take_act8("y8", a->y8, rows, cols, false, &p.y8, s, &n));
  if (a->h8.codes) DPOPT_TRY(take_act8("h8", a->h8, rows, cols, false, &p.h8, s, &n));
  const int64_t gates = gate_count(rows, a->gate_rows);
  if (a->gate.data)
    DPOPT_TRY(take_matrix("gate", a->gate, gates, cols, ps, false, &p.gate, s, &n));
  if (a->dgate.data)
    DPOPT_TRY(take_matrix("dgate", a->dgate, gates, cols, ps, true, &p.dgate, s, &n));
  Mat dummy;
  auto vec = [&](const char* name, const void* q, int64_t len, int64_t size, bool w) {
    return q ? take_matrix(name, dpopt_matrix{const_cast<void*>(q), len}, 1, len, size, w, &dummy,
                           s, &n)
             : DPOPT_OK;
  };
  DPOPT_TRY(vec("w_post", a->w_post, cols, ps, false));
  DPOPT_TRY(vec("w_pre", a->w_pre, cols, ps, false));
  DPOPT_TRY(vec("rstd_post", a->rstd_post, rows, 4, false));
  DPOPT_TRY(vec("rstd_pre", a->rstd_pre, rows, 4, false));
  DPOPT_TRY(vec("dw_post", a->dw_post, cols, ps, true));
  DPOPT_TRY(vec("dw_pre", a->dw_pre, cols, ps, true));
  int64_t need = 0;
  DPOPT_TRY(dpopt_block_join_scratch_bytes(rows, cols, a->gate_rows, &need));
  if (need > 0) {
    if (!a->scratch || (uintptr_t)a->scratch % 256)
      return fail(DPOPT_ERR_INVALID_ARG, "scratch must be non-null and 256-byte aligned");
    if (a->scratch_bytes < need)
      return fail(DPOPT_ERR_INVALID_ARG, "scratch holds %lld bytes, %lld are needed",
                  (long long)a->scratch_bytes, (long long)need);
    DPOPT_TRY(vec("scratch", a->scratch, need, 1, true));
  }
  DPOPT_TRY(check_overlaps(s, n));
  p.rows = rows;
  p.cols = cols;
  p.groups = round_groups(cols);
  p.param_dtype = a->param_dtype;
  p.res_scale = a->res_scale;
  p.branch_scale = a->branch_scale;
  p.gate_rows = a->gate_rows;
  p.w_post = a->w_post;
  p.w_pre = a->w_pre;
  p.rstd_post = a->rstd_post;
  p.rstd_pre = a->rstd_pre;
  p.dw_post = a->dw_post;
  p.dw_pre = a->dw_pre;
  p.partial = static_cast<float*>(a->scratch);
  p.dbg = make_dbg();
  const int64_t parts = part_count(rows);
  if (rows > 0) {
    auto kern = a->dtype == DPOPT_GRAD_BF16  ? block_join_grad_kernel<bf16>
                : a->dtype == DPOPT_GRAD_F16 ? block_join_grad_kernel<fp16>
                                             : block_join_grad_kernel<float>;
    const size_t smem = (size_t)p.groups * 8 * 3 * sizeof(float);
    DPOPT_TRY(allow_smem(kern, smem));
    DPOPT_TRY(launched(
        launch_pdl(kern, (unsigned)parts, kJoinThreads, smem, (cudaStream_t)stream, p),
        "block join gradient"));
  }
  if (!p.dw_pre && !p.dw_post && !p.dgate.data) return DPOPT_OK;
  // gate rows that cross a part's border: one for all rows, or at most one per
  // border (none when the parts are whole numbers of gate rows)
  unsigned gate_sums = 0;
  if (p.dgate.data) {
    if (a->gate_rows == 0)
      gate_sums = rows == 0 || parts > 1;
    else if (rows > 0 && part_rows(rows) % a->gate_rows != 0)
      gate_sums = (unsigned)(parts - 1);
  }
  if (!p.dw_pre && !p.dw_post && gate_sums == 0) return DPOPT_OK;
  const dim3 grid((unsigned)((cols + 31) / 32), 2 + gate_sums);
  return launched(launch_pdl(block_join_finish_kernel, grid, dim3(32 * kFinishRuns), 0,
                             (cudaStream_t)stream, p),
                  "block join gradient sums");
}

}  // extern "C"
