// token_logprob.cu -- log probabilities of given tokens with entropy and top
// alternatives, and their gradient; the formulas stand in include/dpopt.h.
#include <cmath>

#include "ops.cuh"

namespace dpopt {
namespace {

constexpr int kTokThreads = 256;
constexpr int kTokWarps = kTokThreads / 32;

struct LogprobParams {
  int64_t rows, vocab, ld;
  const void* logits;
  const int64_t* tokens;
  int n_tokens, top;
  float inv_temp;
  float *logprob, *stats, *entropy, *top_logprob;
  int64_t* top_index;
  Dbg dbg;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Total order of (logit, index): larger logits first, among equals the lower
// index, a NaN above every number.  -0 counts as +0.
__device__ __forceinline__ uint64_t rank_key(float x, uint32_t index) {
  uint32_t b = __float_as_uint(x + 0.f);
  b = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  if (x != x) b = 0xffffffffu;
  return (uint64_t)b << 32 | (0xffffffffu - index);
}

template <class F>
__device__ __forceinline__ float cta_reduce(float x, float* slot, F f) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = f(x, __shfl_xor_sync(0xffffffffu, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = x;
  __syncthreads();
  x = slot[0];
  for (int w = 1; w < kTokWarps; ++w) x = f(x, slot[w]);
  return x;
}

// One CTA per row.
template <class T>
__global__ void __launch_bounds__(kTokThreads) token_logprob_kernel(const LogprobParams p) {
  pdl_enter();
  __shared__ float slot[kTokWarps];
  __shared__ uint64_t kslot[kTokWarps];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;
    float m = -INFINITY;
    for (int64_t j = threadIdx.x; j < p.vocab; j += kTokThreads) m = max_nan(m, to_f32(x[j]));
    m = cta_reduce(m, slot, [](float a, float b) { return max_nan(a, b); });
    float sum = 0.f, ent = 0.f;
    const bool empty = m == -INFINITY;
    if (!empty) {
      for (int64_t j = threadIdx.x; j < p.vocab; j += kTokThreads) {
        const float s = (to_f32(x[j]) - m) * p.inv_temp;
        const float e = expf(s);
        sum += e;
        if (s != -INFINITY) ent = fmaf(e, s, ent);
      }
    }
    auto add = [](float a, float b) { return a + b; };
    sum = cta_reduce(sum, slot, add);
    ent = cta_reduce(ent, slot, add);
    const float logsum = empty ? 0.f : logf(sum);
    auto logp = [&](float v) {
      return empty ? -INFINITY : (v - m) * p.inv_temp - logsum;
    };
    if (threadIdx.x == 0) {
      p.stats[row * 2] = m;
      p.stats[row * 2 + 1] = logsum;
      if (p.entropy) p.entropy[row] = empty ? 0.f : logsum - ent / sum;
    }
    if ((int)threadIdx.x < p.n_tokens) {
      const int64_t tok = p.tokens[row * p.n_tokens + threadIdx.x];
      p.logprob[row * p.n_tokens + threadIdx.x] =
          tok < 0 ? 0.f : tok >= p.vocab ? NAN : logp(to_f32(x[tok]));
    }
    uint64_t last = ~0ull;
    for (int k = 0; k < p.top; ++k) {
      uint64_t best = 0;
      for (int64_t j = threadIdx.x; j < p.vocab; j += kTokThreads) {
        const uint64_t key = rank_key(to_f32(x[j]), (uint32_t)j);
        if (key < last && key > best) best = key;
      }
      for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
      __syncthreads();
      if ((threadIdx.x & 31) == 0) kslot[threadIdx.x >> 5] = best;
      __syncthreads();
      for (int w = 0; w < kTokWarps; ++w) best = max(best, kslot[w]);
      last = best;
      const uint32_t j = 0xffffffffu - (uint32_t)best;
      if (threadIdx.x == 0 && dbg_ok(p.dbg, j < p.vocab)) {
        p.top_index[row * p.top + k] = j;
        p.top_logprob[row * p.top + k] = logp(to_f32(x[j]));
      }
    }
  }
}

struct LogprobGradParams {
  int64_t rows, vocab, ld, ld_out;
  const void* logits;
  const int64_t* tokens;
  int n_tokens;
  float inv_temp;
  const float *stats, *dlogprob, *entropy, *dentropy;
  const LossScaleState* loss_scale;
  void* dlogits;
  Dbg dbg;
};

// One CTA per row.  Every element gets its share of -p_j; after a barrier the
// given tokens' elements, whose logits were read before (dlogits may be the
// logits), are stored again with their own terms.
template <class T>
__global__ void __launch_bounds__(kTokThreads)
token_logprob_grad_kernel(const LogprobGradParams p) {
  pdl_enter();
  __shared__ int64_t tok[DPOPT_MAX_TOKENS];
  __shared__ float dlp[DPOPT_MAX_TOKENS];
  __shared__ T given[DPOPT_MAX_TOKENS];
  const float scale = (p.loss_scale ? p.loss_scale->scale : 1.f) * p.inv_temp;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;
    T* out = static_cast<T*>(p.dlogits) + row * p.ld_out;
    __syncthreads();
    if ((int)threadIdx.x < p.n_tokens) {
      const int64_t t = p.tokens[row * p.n_tokens + threadIdx.x];
      tok[threadIdx.x] = t;
      dlp[threadIdx.x] = t < 0 ? 0.f : t >= p.vocab ? NAN : p.dlogprob[row * p.n_tokens + threadIdx.x];
      if (t >= 0 && t < p.vocab) given[threadIdx.x] = x[t];
    }
    __syncthreads();
    float a = 0.f;
    for (int i = 0; i < p.n_tokens; ++i) a += dlp[i];
    const float m = p.stats[row * 2], logsum = p.stats[row * 2 + 1];
    const float dh = p.dentropy ? p.dentropy[row] : 0.f;
    const float ent = p.dentropy ? p.entropy[row] : 0.f;
    const bool empty = m == -INFINITY;
    // the gradient of one logit whose own tokens add `own`
    auto grad = [&](float v, float own) {
      const float lp = (v - m) * p.inv_temp - logsum;
      const float e = expf(lp);
      if (empty || v == -INFINITY) return 0.f;
      // e = 0: lp may be so large that its product with dh overflows, or overflow itself
      return scale * (own - (e == 0.f ? 0.f : e * fmaf(dh, lp + ent, a)));
    };
    for (int64_t j = threadIdx.x; j < p.vocab; j += kTokThreads)
      out[j] = from_f32<T>(grad(to_f32(x[j]), 0.f));
    __syncthreads();
    if ((int)threadIdx.x < p.n_tokens) {
      const int64_t t = tok[threadIdx.x];
      bool mine = t >= 0 && t < p.vocab;
      float own = 0.f;
      for (int i = 0; i < p.n_tokens; ++i)
        if (tok[i] == t) {
          if (i < (int)threadIdx.x) mine = false;  // an equal token before this one stores it
          own += dlp[i];
        }
      if (mine && dbg_ok(p.dbg, t < p.vocab))
        out[t] = from_f32<T>(grad(to_f32(given[threadIdx.x]), own));
    }
  }
}

int check_logits(int dtype, int64_t rows, int64_t vocab, int n_tokens, float inv_temperature) {
  if (rows < 0) return fail(DPOPT_ERR_INVALID_ARG, "rows must be >= 0");
  if (vocab < 1) return fail(DPOPT_ERR_INVALID_ARG, "vocab must be >= 1");
  if (vocab >= ((int64_t)1 << 31)) return fail(DPOPT_ERR_UNSUPPORTED, "vocab must be below 2^31");
  if (!known_dtype(dtype)) return fail(DPOPT_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (n_tokens < 0 || n_tokens > DPOPT_MAX_TOKENS)
    return fail(DPOPT_ERR_INVALID_ARG, "n_tokens must lie in [0, %d]", DPOPT_MAX_TOKENS);
  if (!std::isfinite(inv_temperature) || inv_temperature <= 0.f)
    return fail(DPOPT_ERR_INVALID_ARG, "inv_temperature must be finite, > 0");
  return DPOPT_OK;
}

}  // namespace
}  // namespace dpopt

using namespace dpopt;

extern "C" {

int dpopt_token_logprob_scratch_bytes(int64_t rows, int64_t vocab, int top, int64_t* bytes_out) {
  if (!bytes_out) return fail(DPOPT_ERR_INVALID_ARG, "bytes_out is null");
  DPOPT_TRY(check_logits(DPOPT_GRAD_F32, rows, vocab, 0, 1.f));
  if (top < 0 || top > DPOPT_MAX_TOP || top > vocab)
    return fail(DPOPT_ERR_INVALID_ARG, "top must lie in [0, min(vocab, %d)]", DPOPT_MAX_TOP);
  *bytes_out = 0;
  return DPOPT_OK;
}

int dpopt_token_logprob(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                        const int64_t* tokens, int n_tokens, float inv_temperature,
                        float* logprob, float* stats, float* entropy, int top,
                        float* top_logprob, int64_t* top_index, void* scratch,
                        int64_t scratch_bytes, dpopt_stream_t stream) {
  DPOPT_TRY(check_logits(dtype, rows, vocab, n_tokens, inv_temperature));
  int64_t need = 0;
  DPOPT_TRY(dpopt_token_logprob_scratch_bytes(rows, vocab, top, &need));
  if (rows == 0) return DPOPT_OK;
  Span s[8];
  int n = 0;
  Mat x, dummy;
  auto take = [&](const char* name, const void* q, int64_t per_row, int64_t size, bool w) {
    return take_matrix(name, dpopt_matrix{const_cast<void*>(q), rows * per_row}, 1, rows * per_row,
                       size, w, &dummy, s, &n);
  };
  DPOPT_TRY(take_matrix("logits", dpopt_matrix{const_cast<void*>(logits), ld}, rows, vocab,
                        dtype_size(dtype), false, &x, s, &n));
  if (n_tokens > 0) {
    DPOPT_TRY(take("tokens", tokens, n_tokens, 8, false));
    DPOPT_TRY(take("logprob", logprob, n_tokens, 4, true));
  }
  DPOPT_TRY(take("stats", stats, 2, 4, true));
  if (entropy) DPOPT_TRY(take("entropy", entropy, 1, 4, true));
  if (top > 0) {
    DPOPT_TRY(take("top_logprob", top_logprob, top, 4, true));
    DPOPT_TRY(take("top_index", top_index, top, 8, true));
  }
  if (need > 0) {
    if (!scratch || (uintptr_t)scratch % 256)
      return fail(DPOPT_ERR_INVALID_ARG, "scratch must be non-null and 256-byte aligned");
    if (scratch_bytes < need)
      return fail(DPOPT_ERR_INVALID_ARG, "scratch holds %lld bytes, %lld are needed",
                  (long long)scratch_bytes, (long long)need);
    DPOPT_TRY(take_matrix("scratch", dpopt_matrix{scratch, need}, 1, need, 1, true, &dummy, s, &n));
  }
  DPOPT_TRY(check_overlaps(s, n));
  LogprobParams p{rows,     vocab, x.ld,    logits,  tokens,      n_tokens,  top,
                  inv_temperature, logprob, stats,   entropy,     top_logprob, top_index, make_dbg()};
  int sms = 0;
  DPOPT_TRY(sm_count(&sms));
  auto kern = dtype == DPOPT_GRAD_BF16  ? token_logprob_kernel<bf16>
              : dtype == DPOPT_GRAD_F16 ? token_logprob_kernel<fp16>
                                        : token_logprob_kernel<float>;
  const unsigned grid = (unsigned)std::min<int64_t>(rows, (int64_t)sms * 8);
  return launched(launch_pdl(kern, grid, kTokThreads, 0, (cudaStream_t)stream, p),
                  "token logprob");
}

int dpopt_token_logprob_backward(const void* logits, int dtype, int64_t rows, int64_t vocab,
                                 int64_t ld, const int64_t* tokens, int n_tokens,
                                 float inv_temperature, const float* stats, const float* dlogprob,
                                 const float* entropy, const float* dentropy,
                                 const dpopt_loss_scale_state* loss_scale, void* dlogits,
                                 int64_t ld_dlogits, dpopt_stream_t stream) {
  DPOPT_TRY(check_logits(dtype, rows, vocab, n_tokens, inv_temperature));
  if ((entropy != nullptr) != (dentropy != nullptr))
    return fail(DPOPT_ERR_INVALID_ARG, "entropy and dentropy must be given together");
  if ((uintptr_t)loss_scale % 8)
    return fail(DPOPT_ERR_INVALID_ARG, "loss_scale must be 8-byte aligned");
  if (rows == 0) return DPOPT_OK;
  Span s[8];
  int n = 0;
  Mat x, d, dummy;
  auto take = [&](const char* name, const void* q, int64_t per_row, int64_t size) {
    return take_matrix(name, dpopt_matrix{const_cast<void*>(q), rows * per_row}, 1, rows * per_row,
                       size, false, &dummy, s, &n);
  };
  const int64_t es = dtype_size(dtype);
  DPOPT_TRY(take_matrix("logits", dpopt_matrix{const_cast<void*>(logits), ld}, rows, vocab, es,
                        false, &x, s, &n));
  DPOPT_TRY(take_matrix("dlogits", dpopt_matrix{dlogits, ld_dlogits}, rows, vocab, es, true, &d, s,
                        &n));
  if (logits == dlogits && (rows <= 1 || ld == ld_dlogits)) s[0].hi = s[0].lo;  // in place
  if (n_tokens > 0) {
    DPOPT_TRY(take("tokens", tokens, n_tokens, 8));
    DPOPT_TRY(take("dlogprob", dlogprob, n_tokens, 4));
  }
  DPOPT_TRY(take("stats", stats, 2, 4));
  if (dentropy) {
    DPOPT_TRY(take("entropy", entropy, 1, 4));
    DPOPT_TRY(take("dentropy", dentropy, 1, 4));
  }
  if (loss_scale)
    DPOPT_TRY(take_matrix("loss_scale",
                          dpopt_matrix{const_cast<dpopt_loss_scale_state*>(loss_scale), 32}, 1,
                          sizeof(dpopt_loss_scale_state), 1, false, &dummy, s, &n));
  DPOPT_TRY(check_overlaps(s, n));
  LogprobGradParams p{rows,  vocab,    x.ld,    d.ld,     logits,
                      tokens, n_tokens, inv_temperature, stats, dlogprob,
                      entropy, dentropy, reinterpret_cast<const LossScaleState*>(loss_scale),
                      dlogits, make_dbg()};
  int sms = 0;
  DPOPT_TRY(sm_count(&sms));
  auto kern = dtype == DPOPT_GRAD_BF16  ? token_logprob_grad_kernel<bf16>
              : dtype == DPOPT_GRAD_F16 ? token_logprob_grad_kernel<fp16>
                                        : token_logprob_grad_kernel<float>;
  const unsigned grid = (unsigned)std::min<int64_t>(rows, (int64_t)sms * 8);
  return launched(launch_pdl(kern, grid, kTokThreads, 0, (cudaStream_t)stream, p),
                  "token logprob gradient");
}

}  // extern "C"
