// act8_wgrad.cu -- weight gradient of a linear layer from its packed input:
// dw[i][j] = sum_t dy[t][i] * value(t, j) (+ addend).
#include "ops.cuh"

namespace dpopt {
namespace {

struct WgradParams {
  int64_t tokens, n, k;
  Mat dy;
  Act8Out x;
  Mat dw, addend;
  int out_dtype;
  Dbg dbg;
};

// 64 x 64 outputs per CTA, 4 x 4 per thread, 16 tokens at a time in shared
// memory: any size, stride and alignment.
constexpr int kTile = 64, kDepth = 16, kWgradThreads = 256;

template <class T>
__global__ void __launch_bounds__(kWgradThreads) act8_wgrad_kernel(const WgradParams p) {
  pdl_enter();
  __shared__ float a[kDepth][kTile], b[kDepth][kTile];
  const int64_t i0 = (int64_t)blockIdx.y * kTile, j0 = (int64_t)blockIdx.x * kTile;
  const int ti = threadIdx.x / 16 * 4, tj = threadIdx.x % 16 * 4;
  float acc[4][4] = {};
  for (int64_t t0 = 0; t0 < p.tokens; t0 += kDepth) {
    __syncthreads();
    for (int e = threadIdx.x; e < kDepth * kTile; e += kWgradThreads) {
      const int64_t t = t0 + e / kTile;
      const int c = e % kTile;
      float va = 0.f, vb = 0.f;
      if (t < p.tokens && i0 + c < p.n)
        va = to_f32(static_cast<const T*>(p.dy.data)[t * p.dy.ld + i0 + c]);
      if (t < p.tokens && j0 + c < p.k)
        vb = (float)p.x.codes[t * p.x.ld_codes + j0 + c] *
             act8_scale(p.x.exps[t * p.x.ld_exps + (j0 + c) / kAct8Block]);
      a[e / kTile][c] = va;
      b[e / kTile][c] = vb;
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kDepth; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[t][ti + i], b[t][tj + j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = i0 + ti + i, c = j0 + tj + j;
      if (r >= p.n || c >= p.k) continue;
      float v = acc[i][j];
      if (p.addend.data) v += ld_any(p.addend.data, p.out_dtype, r * p.addend.ld + c);
      st_any(p.dw.data, p.out_dtype, r * p.dw.ld + c, v);
    }
}

}  // namespace
}  // namespace dpopt

using namespace dpopt;

extern "C" {

int dpopt_act8_wgrad_scratch_bytes(int64_t tokens, int64_t n, int64_t k, int64_t* bytes_out) {
  if (!bytes_out || tokens < 0 || n < 0 || k < 0)
    return fail(DPOPT_ERR_INVALID_ARG, "wgrad scratch: null output or a negative size");
  *bytes_out = 0;
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
  const int64_t limit = (int64_t)1 << 31;
  if (tokens >= limit || n >= limit || k >= limit)
    return fail(DPOPT_ERR_UNSUPPORTED, "sizes must be below 2^31");
  if (n == 0 || k == 0) return DPOPT_OK;
  WgradParams p{};
  Span s[8];
  int cnt = 0;
  Mat dummy;
  const int64_t es = dtype_size(dtype), os = dtype_size(out_dtype);
  DPOPT_TRY(take_matrix("dw", dpopt_matrix{dw, ld_dw}, n, k, os, true, &p.dw, s, &cnt));
  if (addend) {
    DPOPT_TRY(take_matrix("addend", dpopt_matrix{const_cast<void*>(addend), ld_addend}, n, k, os,
                          false, &p.addend, s, &cnt));
    if (addend == dw && (n == 1 || ld_addend == ld_dw)) s[1].hi = s[1].lo;  // in place
  }
  DPOPT_TRY(take_matrix("dy", dpopt_matrix{const_cast<void*>(dy), ld_dy}, tokens, n, es, false,
                        &p.dy, s, &cnt));
  DPOPT_TRY(take_act8("the packed input",
                      dpopt_act8{const_cast<int8_t*>(codes), ld_codes,
                                 const_cast<uint8_t*>(exps), ld_exps},
                      tokens, k, false, &p.x, s, &cnt));
  int64_t need = 0;
  DPOPT_TRY(dpopt_act8_wgrad_scratch_bytes(tokens, n, k, &need));
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
  p.tokens = tokens;
  p.n = n;
  p.k = k;
  p.out_dtype = out_dtype;
  p.dbg = make_dbg();
  const int64_t gy = (n + kTile - 1) / kTile;
  if (gy > 65535) return fail(DPOPT_ERR_UNSUPPORTED, "n %lld is too large", (long long)n);
  const dim3 grid((unsigned)((k + kTile - 1) / kTile), (unsigned)gy);
  auto kern = dtype == DPOPT_GRAD_BF16 ? act8_wgrad_kernel<bf16> : act8_wgrad_kernel<fp16>;
  return launched(launch_pdl(kern, grid, kWgradThreads, 0, (cudaStream_t)stream, p),
                  "act8 weight gradient");
}

}  // extern "C"
