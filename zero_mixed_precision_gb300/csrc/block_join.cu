// block_join.cu -- the join between two transformer blocks (the norm after the
// block, gate, residual scale, the norm before the next block) and its
// gradient; the formulas stand in include/dpopt.h.
#include <cmath>

#include "ops.cuh"

namespace dpopt {
namespace {

// A row is held by one CTA of tpr threads (a multiple of 32), in NV fragments of 8
// columns per thread: as few as 512 threads can cover the row with.  In the
// vector form (VEC: every matrix may be moved 16 bytes at a time) thread t's
// fragment v is the columns (v tpr + t) 8 .. + 7; in the element form, for odd
// widths and alignments, its element i is column (v 8 + i) tpr + t, so that a
// warp always touches neighbouring columns.  Either way a block of 32 columns
// lies in one warp.  The row index depends on blockIdx alone, which keeps the
// row addresses out of the threads' registers.
constexpr int kJoinCta = 512, kJoinSms = 152;

struct JoinParams {
  int64_t rows;
  int cols, tpr, param_dtype;
  float eps, res_scale, branch_scale;
  int64_t gate_rows;
  Mat h, y, gate, h_out, u;
  const void *w_post, *w_pre;
  float *rstd_post, *rstd_pre;
  Act8Out y8, h8, u8;
  Dbg dbg;
};

__host__ __device__ inline int row_frags(int64_t cols) { return cols <= 8 * kJoinCta ? 1 : cols <= 16 * kJoinCta ? 2 : 4; }
__host__ __device__ inline int row_threads(int64_t cols) {
  const int64_t per_warp = 256 * row_frags(cols);
  return (int)((cols + per_warp - 1) / per_warp) * 32;
}

// Sum of N values over a CTA, the same bits in each thread: the warps'
// butterflies, then the warps' sums in warp order (or as a butterfly).  Callers
// alternate between two slot arrays, so that one barrier is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&x)[N], float (*slot)[N], int tpr) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = warp_sum(x[i]);
  if (tpr == 32) return;
  const int warps = tpr >> 5, lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) slot[threadIdx.x >> 5][i] = x[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (warps <= 4) {
      x[i] = slot[0][i];
      for (int w = 1; w < warps; ++w) x[i] += slot[w][i];
    } else {
      const int w = lane & (kJoinCta / 32 - 1);  // both halves of the warp alike
      x[i] = w < warps ? slot[w][i] : 0.f;
#pragma unroll
      for (int o = kJoinCta / 64; o > 0; o >>= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    }
  }
}

// Values of a parameter (row `at` elements in; ones where it is absent) at a
// thread's columns, into its places out[i * stride].  Not inlined: parameters are
// read once per launch or gate row, and their three types and eight addresses
// would take the registers of the loops around it.
template <bool VEC, int NV>
__device__ __noinline__ void stage_param(const void* w, int dtype, int64_t at, int t, int tpr,
                                         int cols, float* out, int stride) {
#pragma unroll 1
  for (int v = 0; v < NV; ++v)
#pragma unroll 4
    for (int i = 0; i < 8; ++i) {
      const int c = column<VEC>(v, i, t, tpr);
      out[(v * 8 + i) * stride] = w && c < cols ? ld_any(w, dtype, at + c) : 1.f;
    }
}

__device__ __forceinline__ int64_t gate_row_of(int64_t gate_rows, int64_t row) {
  return gate_rows > 0 ? row / gate_rows : 0;
}

// A CTA walks rows; the next row's h and y are loaded before the present row's
// two sums, and h_out stays in registers in fp32 between the norms.  The
// parameters are kept as branch_scale * gate * w_post and w_pre.
template <class T, bool VEC, int NV>
__global__ void __launch_bounds__(kJoinCta, NV == 1 ? 2 : 1)
    block_join_kernel(const __grid_constant__ JoinParams p) {
  pdl_enter();
  __shared__ float slot[2][kJoinCta / 32][1];
  extern __shared__ float stage[];  // 8 NV places per thread
  const int t = threadIdx.x, tpr = blockDim.x;
  const int cols = p.cols;
  if (!dbg_ok(p.dbg, tpr * 8 * NV >= cols)) return;
  const float inv_c = 1.f / (float)cols;
  float* mine = stage + t;
  float pb[NV][8], wpre[NV][8];
  stage_param<VEC, NV>(p.w_pre, p.param_dtype, 0, t, tpr, cols, mine, tpr);
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) wpre[v][i] = mine[(v * 8 + i) * tpr];
  Frag<T, VEC> fh[NV], fy[NV];
  int64_t row = blockIdx.x;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    fh[v].load(p.h, row, v, t, tpr, cols);
    fy[v].load(p.y, row, v, t, tpr, cols);
  }
  int64_t held = -1;  // gate row in pb
  for (; row < p.rows; row += gridDim.x) {
    const int64_t grow = gate_row_of(p.gate_rows, row);
    if (grow != held) {
      held = grow;
      stage_param<VEC, NV>(p.w_post, p.param_dtype, 0, t, tpr, cols, mine, tpr);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) pb[v][i] = p.branch_scale * mine[(v * 8 + i) * tpr];
      if (p.gate.data) {
        stage_param<VEC, NV>(p.gate.data, p.param_dtype, grow * p.gate.ld, t, tpr, cols, mine,
                             tpr);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i) pb[v][i] *= mine[(v * 8 + i) * tpr];
      }
    }
    float h[NV][8], y[NV][8];
    const int64_t next = row + gridDim.x;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      fh[v].widen(h[v]);
      fy[v].widen(y[v]);
      if (next < p.rows) {
        fh[v].load(p.h, next, v, t, tpr, cols);
        fy[v].load(p.y, next, v, t, tpr, cols);
      }
    }
    float rpost = 1.f;
    if (p.rstd_post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(y[v][i], y[v][i], ss[0]);
      row_sum<1>(ss, slot[0], tpr);
      rpost = rsqrtf(fmaf(ss[0], inv_c, p.eps));
      if (t == 0) p.rstd_post[row] = rpost;
    }
    float ss[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (p.y8.codes) frag_pack<T, VEC>(p.y8, row, v, t, tpr, cols, y[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[v][i] = fmaf(pb[v][i], y[v][i] * rpost, p.res_scale * h[v][i]);
        ss[0] = fmaf(h[v][i], h[v][i], ss[0]);
      }
      frag_store<T, VEC>(p.h_out, row, v, t, tpr, cols, h[v]);
      if (p.h8.codes) {
        float r[8];
        round8<T>(h[v], r);
        frag_pack<T, VEC>(p.h8, row, v, t, tpr, cols, r);
      }
    }
    if (!p.u.data) {
      __syncthreads();  // the only sum's slots are used again in the next row
      continue;
    }
    row_sum<1>(ss, slot[1], tpr);
    const float rpre = rsqrtf(fmaf(ss[0], inv_c, p.eps));
    if (t == 0) p.rstd_pre[row] = rpre;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] *= rpre * wpre[v][i];
      frag_store<T, VEC>(p.u, row, v, t, tpr, cols, h[v]);
      if (p.u8.codes) {
        float r[8];
        round8<T>(h[v], r);
        frag_pack<T, VEC>(p.u8, row, v, t, tpr, cols, r);
      }
    }
    if (!p.rstd_post) __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------

// Sums over rows: the rows are cut into runs, whose number and borders depend on
// the sizes alone (as many as 152 SMs hold CTAs at a time, but no run of fewer
// than kPartMinRows rows when there are more rows than SMs).  Each run's CTA leaves one partial row per sum in scratch and the finish kernel adds them
// in order, so the result does not depend on the GPU or on timing.
constexpr int kPartMinRows = 4;

// CTAs of the gradient's kernel an SM holds (its registers are sized for kJoinCta
// threads).
__host__ __device__ inline int ctas_per_sm(int64_t cols) {
  const int n = kJoinCta / row_threads(cols);
  return n < 1 ? 1 : n;
}
__host__ __device__ inline int64_t part_rows(int64_t rows, int64_t cols) {
  const int64_t at_once = (int64_t)kJoinSms * ctas_per_sm(cols);
  const int64_t each = (rows + at_once - 1) / at_once;
  return each < kPartMinRows && rows > kJoinSms ? kPartMinRows : each < 1 ? 1 : each;
}
__host__ __device__ inline int64_t part_count(int64_t rows, int64_t cols) {
  return (rows + part_rows(rows, cols) - 1) / part_rows(rows, cols);
}

// Partial rows of one part: dw_pre, dw_post, and up to two of dgate (of the
// part's first gate row, and of its last when that is another one; gate rows
// that lie inside a part are stored at once).
enum { kPartWPre = 0, kPartWPost = 1, kPartGateFirst = 2, kPartGateLast = 3, kPartSlots = 4 };

struct JoinGradParams {
  int64_t rows, per, parts;  // rows of a part, parts
  int cols, width, tpr;      // width: cols rounded up to whole blocks
  // the vector form's ring in shared memory: rows held, bytes of one, and where and
  // how large the fragments of each array are (enum kIn*)
  int stages;
  uint32_t stage_bytes, frag_at[4], frag_bytes[4];
  int param_dtype;
  float res_scale, branch_scale;
  int64_t gate_rows;
  Mat dh_out, du, y, h_out, gate, dh, dy, dgate;
  Act8Out y8, h8;
  const void *w_post, *w_pre;
  const float *rstd_post, *rstd_pre;
  void *dw_post, *dw_pre;
  float* partial;  // [part][kPartSlots][width]
  Dbg dbg;
};

__device__ __forceinline__ float* part_row(const JoinGradParams& p, int64_t part, int slot) {
  return p.partial + (part * kPartSlots + slot) * p.width;
}

// Rows [lo, hi) that use the gate row of `row`.
__host__ __device__ inline void gate_span(int64_t gate_rows, int64_t rows, int64_t row, int64_t* lo,
                                          int64_t* hi) {
  *lo = gate_rows > 0 ? row / gate_rows * gate_rows : 0;
  *hi = gate_rows > 0 && *lo + gate_rows < rows ? *lo + gate_rows : rows;
}

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// The four arrays a gradient row reads, as a thread gets at its fragments.
// Vector form: a ring of rows in shared memory, each thread copying (cp.async) and
// reading only its own fragments, so that rows are in flight without registers
// and without barriers.  Element form: straight from global memory (the second
// reading of a row comes from L1).
enum { kInDh = 0, kInDu = 1, kInY = 2, kInH = 3 };

template <class T, bool VEC, int NV>
struct GradRow {
  const JoinGradParams& p;
  const int t, tpr;
  // this thread's places in a stage of the ring: 16 or 32 bytes a fragment, and 8
  const uint32_t ring;
  uint32_t next[2][NV];  // exponent bytes of y and h of the row after the present one
  float scale[2][NV];    // and the present row's scales

  __device__ __forceinline__ GradRow(const JoinGradParams& q, uint32_t r)
      : p(q), t(threadIdx.x), tpr(blockDim.x), ring(r) {}

  __device__ __forceinline__ const Mat& mat(int which) const {
    return which == kInDh ? p.dh_out : which == kInDu ? p.du : which == kInY ? p.y : p.h_out;
  }
  __device__ __forceinline__ const Act8Out& act(int which) const {
    return which == kInY ? p.y8 : p.h8;
  }
  __device__ __forceinline__ bool packed(int which) const {
    return which == kInY ? p.y8.codes != nullptr : which == kInH && p.h8.codes != nullptr;
  }
  __device__ __forceinline__ bool present(int which) const {
    return which == kInDh || which == kInY || p.du.data != nullptr;
  }
  __device__ __forceinline__ uint32_t slot(uint32_t at, int which, int v) const {
    return at + p.frag_at[which] + (v * tpr + t) * p.frag_bytes[which];
  }

  // Start the copies of a row into the stage at `at`.
  __device__ __forceinline__ void fetch(int64_t row, uint32_t at) const {
    if constexpr (VEC) {
#pragma unroll
      for (int which = 0; which < 4; ++which) {
        if (!present(which)) continue;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int c = column<true>(v, 0, t, tpr);
          if (c >= p.cols) continue;
          if (packed(which)) {
            copy_async8(slot(at, which, v), act(which).codes + row * act(which).ld_codes + c);
          } else {
            const T* src = static_cast<const T*>(mat(which).data) + row * mat(which).ld + c;
            copy_async16(slot(at, which, v), src);
            if constexpr (sizeof(T) == 4) copy_async16(slot(at, which, v) + 16, src + 4);
          }
        }
      }
    }
  }
  // The exponent bytes of a row, asked for one row ahead.
  __device__ __forceinline__ void fetch_scales(int64_t row) {
    if constexpr (VEC) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (packed(kInY + k) && present(kInY + k)) {
          const uint8_t* exps = act(kInY + k).exps + row * act(kInY + k).ld_exps;
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int c = column<true>(v, 0, t, tpr);
            next[k][v] = c < p.cols ? exps[c / kAct8Block] : 0;
          }
        }
    }
  }
  __device__ __forceinline__ void take_scales() {
    if constexpr (VEC) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (packed(kInY + k) && present(kInY + k))
#pragma unroll
          for (int v = 0; v < NV; ++v) scale[k][v] = act8_scale(next[k][v]);
    }
  }

  __device__ __forceinline__ void get(int64_t row, uint32_t at, int which, int v,
                                      float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.f;
    if (!present(which)) return;
    if constexpr (VEC) {
      if (column<true>(v, 0, t, tpr) >= p.cols) return;
      const uint32_t a = slot(at, which, v);
      if (packed(which)) {
        uint2 c;
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(c.x), "=r"(c.y) : "r"(a) : "memory");
        act8_values(c, scale[which - kInY][v], f);
        return;
      }
      Raw8<T> r;
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(r.v.x), "=r"(r.v.y), "=r"(r.v.z), "=r"(r.v.w)
                   : "r"(a)
                   : "memory");
      if constexpr (sizeof(T) == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r.w.x), "=r"(r.w.y), "=r"(r.w.z), "=r"(r.w.w)
                     : "r"(a + 16)
                     : "memory");
      widen8<T>(r, f);
    } else if (packed(which)) {
      const int8_t* codes = act(which).codes + row * act(which).ld_codes;
      const uint8_t* exps = act(which).exps + row * act(which).ld_exps;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = column<false>(v, i, t, tpr);
        if (c < p.cols) f[i] = (float)codes[c] * act8_scale(exps[c / kAct8Block]);
      }
    } else {
      const T* q = static_cast<const T*>(mat(which).data) + row * mat(which).ld;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = column<false>(v, i, t, tpr);
        if (c < p.cols) f[i] = to_f32(q[c]);
      }
    }
  }
};

// At the end of a gate row's rows in a part: its sums branch_scale * e (in `mine`)
// go into dw_post's and into dgate, or into a partial row of it.
template <bool VEC, int NV>
__device__ __noinline__ void close_gate_row(const JoinGradParams& p, int64_t part, int64_t lo,
                                            int64_t hi, int64_t row, bool first_gate, int t,
                                            float* post, const float* mine, int stride) {
  int64_t glo, ghi;
  gate_span(p.gate_rows, p.rows, row, &glo, &ghi);
  const bool inside = glo >= lo && ghi <= hi;
  const int64_t grow = gate_row_of(p.gate_rows, row);
  float* out = part_row(p, part, first_gate ? kPartGateFirst : kPartGateLast);
#pragma unroll 1
  for (int v = 0; v < NV; ++v)
#pragma unroll 4
    for (int i = 0; i < 8; ++i) {
      const int c = column<VEC>(v, i, t, p.tpr);
      if (c >= p.cols) continue;
      const float x = mine[(v * 8 + i) * stride];
      const float g = p.gate.data ? ld_any(p.gate.data, p.param_dtype, grow * p.gate.ld + c) : 1.f;
      const float w = p.w_post ? ld_any(p.w_post, p.param_dtype, c) : 1.f;
      post[(v * 8 + i) * stride] = fmaf(g, x, post[(v * 8 + i) * stride]);
      if (!p.dgate.data) continue;
      if (inside)
        st_any(p.dgate.data, p.param_dtype, grow * p.dgate.ld + c, w * x);
      else
        out[c] = w * x;
    }
}

// One CTA per run of rows.  Per row one reading forms three sums,
//   s = <w_pre du, h>,  a = <q, dh_out + r1 w_pre du>,  b = <q, h>,
//   q = branch_scale w_post gate y,
// from which <w_post dz, y> = a - r1^3 s / C b; a second reading forms the outputs.
// Sums over rows per column: dw_pre, and e = sum d y rstd_post, from which, while
// the gate row stays the same, dw_post grows by branch gate e and dgate is branch
// w_post e.
template <class T, bool VEC, int NV>
__global__ void __launch_bounds__(kJoinCta, 1)
    block_join_grad_kernel(const __grid_constant__ JoinGradParams p) {
  pdl_enter();
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ float slot[2][kJoinCta / 32][3];
  const int t = threadIdx.x, tpr = blockDim.x;
  const int64_t lo = blockIdx.x * p.per, hi = min(p.rows, lo + p.per);
  if (!dbg_ok(p.dbg, tpr * 8 * NV >= p.cols && lo < hi)) return;
  const float inv_c = 1.f / (float)p.cols;
  // dw_post of finished gate rows, and parameters and sums on their way: one
  // place per column of a thread
  float* post = reinterpret_cast<float*>(dyn) + t;
  float* mine = post + 8 * NV * tpr;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(dyn) + 16 * NV * tpr * 4;
  GradRow<T, VEC, NV> in(p, ring);
  float wpre[NV][8], q[NV][8], acc[NV][8], e[NV][8];
  stage_param<VEC, NV>(p.w_pre, p.param_dtype, 0, t, tpr, p.cols, mine, tpr);
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      wpre[v][i] = mine[(v * 8 + i) * tpr];
      acc[v][i] = e[v][i] = 0.f;
      post[(v * 8 + i) * tpr] = 0.f;
    }
  for (int s = 0; s < p.stages; ++s) {
    if (lo + s < hi) in.fetch(lo + s, ring + s * p.stage_bytes);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  in.fetch_scales(lo);
  int64_t held = -1;
  bool first_gate = true;
  int stage = 0;
  for (int64_t row = lo; row < hi; ++row) {
    const int64_t grow = gate_row_of(p.gate_rows, row);
    if (grow != held) {
      held = grow;
      stage_param<VEC, NV>(p.w_post, p.param_dtype, 0, t, tpr, p.cols, mine, tpr);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) q[v][i] = p.branch_scale * mine[(v * 8 + i) * tpr];
      if (p.gate.data) {
        stage_param<VEC, NV>(p.gate.data, p.param_dtype, grow * p.gate.ld, t, tpr, p.cols, mine,
                             tpr);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int i = 0; i < 8; ++i) q[v][i] *= mine[(v * 8 + i) * tpr];
      }
    }
    const float r1 = p.du.data ? p.rstd_pre[row] : 0.f;
    const float r2 = p.rstd_post ? p.rstd_post[row] : 1.f;
    in.take_scales();
    if (row + 1 < hi) in.fetch_scales(row + 1);
    const uint32_t at = ring + stage * p.stage_bytes;
    if constexpr (VEC) {
      // the oldest of the rows asked for has arrived
      if (p.stages == 1)
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      else if (p.stages == 2)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      else
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    }
    float sum[3];
    {
      uint64_t s2 = 0, a2 = 0, b2 = 0;
      const uint64_t rr = pair(r1, r1);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float d[8], u[8], h[8], y[8];
        in.get(row, at, kInDh, v, d);
        in.get(row, at, kInDu, v, u);
        in.get(row, at, kInY, v, y);
        in.get(row, at, kInH, v, h);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const uint64_t wu = mul2(pair(wpre[v][i], wpre[v][i + 1]), pair(u[i], u[i + 1]));
          const uint64_t qy = mul2(pair(q[v][i], q[v][i + 1]), pair(y[i], y[i + 1]));
          const uint64_t hh = pair(h[i], h[i + 1]);
          s2 = fma2(wu, hh, s2);
          a2 = fma2(qy, fma2(rr, wu, pair(d[i], d[i + 1])), a2);
          b2 = fma2(qy, hh, b2);
        }
      }
      sum[0] = lane0(s2) + lane1(s2);
      sum[1] = lane0(a2) + lane1(a2);
      sum[2] = lane0(b2) + lane1(b2);
    }
    row_sum<3>(sum, slot[row & 1], tpr);
    const float k1 = r1 * r1 * r1 * sum[0] * inv_c;
    const float k2 = p.rstd_post ? r2 * r2 * r2 * (sum[1] - k1 * sum[2]) * inv_c : 0.f;
    {
      const uint64_t r1p = pair(r1, r1), r2p = pair(r2, r2), k1p = pair(-k1, -k1),
                     k2p = pair(-k2, -k2);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float d[8], u[8], h[8], y[8];
        in.get(row, at, kInDh, v, d);
        in.get(row, at, kInDu, v, u);
        in.get(row, at, kInY, v, y);
        in.get(row, at, kInH, v, h);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const uint64_t u2 = pair(u[i], u[i + 1]), y2 = pair(y[i], y[i + 1]);
          const uint64_t h2 = pair(h[i], h[i + 1]);
          const uint64_t full =
              fma2(k1p, h2, fma2(r1p, mul2(pair(wpre[v][i], wpre[v][i + 1]), u2),
                                 pair(d[i], d[i + 1])));
          const uint64_t fr = mul2(full, r2p);
          const uint64_t ac = fma2(u2, mul2(h2, r1p), pair(acc[v][i], acc[v][i + 1]));
          const uint64_t ee = fma2(fr, y2, pair(e[v][i], e[v][i + 1]));
          const uint64_t dy = fma2(k2p, y2, mul2(pair(q[v][i], q[v][i + 1]), fr));
          acc[v][i] = lane0(ac);
          acc[v][i + 1] = lane1(ac);
          e[v][i] = lane0(ee);
          e[v][i + 1] = lane1(ee);
          d[i] = lane0(full);
          d[i + 1] = lane1(full);
          u[i] = lane0(dy);
          u[i + 1] = lane1(dy);
        }
        if (p.dh.data) {
          if (p.res_scale != 1.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] *= p.res_scale;
          }
          frag_store<T, VEC>(p.dh, row, v, t, tpr, p.cols, d);
        }
        frag_store<T, VEC>(p.dy, row, v, t, tpr, p.cols, u);
      }
    }
    if constexpr (VEC) {
      if (row + p.stages < hi) in.fetch(row + p.stages, at);
      asm volatile("cp.async.commit_group;" ::: "memory");
      stage = stage + 1 == p.stages ? 0 : stage + 1;
    }
    if (row + 1 == hi || gate_row_of(p.gate_rows, row + 1) != grow) {
      // the last row here of its gate row
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          mine[(v * 8 + i) * tpr] = p.branch_scale * e[v][i];
          e[v][i] = 0.f;
        }
      close_gate_row<VEC, NV>(p, blockIdx.x, lo, hi, row, first_gate, t, post, mine, tpr);
      first_gate = false;
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<VEC>(v, i, t, tpr);
      if (c >= p.cols) continue;
      if (p.dw_pre) part_row(p, blockIdx.x, kPartWPre)[c] = acc[v][i];
      if (p.dw_post) part_row(p, blockIdx.x, kPartWPost)[c] = post[(v * 8 + i) * tpr];
    }
}

// Adds the parts' partial rows.  blockIdx.y: 0 dw_pre, 1 dw_post, 2 + q the gate
// row that begins in part q and reaches into part q + 1 (with one gate row
// for all rows, q = 0).  32 columns x 8 runs of parts per CTA; the runs' sums
// are added in order.
constexpr int kFinishRuns = 8;

__global__ void __launch_bounds__(32 * kFinishRuns)
block_join_finish_kernel(const __grid_constant__ JoinGradParams p) {
  pdl_enter();
  __shared__ float run_sum[kFinishRuns][33];
  const int64_t parts = p.parts, per = p.per;
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

int64_t whole_blocks(int64_t cols) {
  return (cols + kAct8Block - 1) / kAct8Block * kAct8Block;
}

bool vec_ok(const Mat& m) { return !m.data || m.vec; }
bool vec_ok(const Act8Out& a) { return !a.codes || a.vec; }

constexpr size_t kJoinSmem = 220 * 1024;  // of 227 KB; the static arrays need some

template <class K>
int allow_smem(K kern, size_t bytes) {
  if (bytes <= 40 * 1024) return DPOPT_OK;  // 48 KB without asking, static arrays included
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  return e == cudaSuccess ? DPOPT_OK : cuda_fail(e, "shared memory size");
}

template <class T, bool VEC, int NV>
int launch_join_at(JoinParams& p, cudaStream_t stream) {
  auto kern = block_join_kernel<T, VEC, NV>;
  int sms = 0, per_sm = 0;
  DPOPT_TRY(sm_count(&sms));
  const size_t smem = (size_t)p.tpr * 8 * NV * sizeof(float);
  DPOPT_TRY(allow_smem(kern, smem));
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, p.tpr, smem);
  if (e != cudaSuccess) return cuda_fail(e, "block join occupancy");
  const unsigned grid =
      (unsigned)std::min<int64_t>(p.rows, (int64_t)sms * std::max(per_sm, 1));
  return launched(launch_pdl(kern, grid, p.tpr, smem, stream, p), "block join");
}

template <class T>
int launch_join(JoinParams& p, bool vec, cudaStream_t stream) {
  switch (row_frags(p.cols)) {
    case 1:
      return vec ? launch_join_at<T, true, 1>(p, stream) : launch_join_at<T, false, 1>(p, stream);
    case 2:
      return vec ? launch_join_at<T, true, 2>(p, stream) : launch_join_at<T, false, 2>(p, stream);
    default:
      return vec ? launch_join_at<T, true, 4>(p, stream) : launch_join_at<T, false, 4>(p, stream);
  }
}

template <class T, bool VEC, int NV>
int launch_join_grad_at(JoinGradParams& p, cudaStream_t stream) {
  auto kern = block_join_grad_kernel<T, VEC, NV>;
  const size_t room = kJoinSmem / ctas_per_sm(p.cols);
  const size_t sums = (size_t)p.tpr * 16 * NV * sizeof(float);
  p.stages = VEC ? (int)std::min<size_t>(3, (room - sums) / p.stage_bytes) : 0;
  const size_t smem = sums + (size_t)p.stages * p.stage_bytes;
  DPOPT_TRY(allow_smem(kern, smem));
  return launched(launch_pdl(kern, (unsigned)p.parts, p.tpr, smem, stream, p),
                  "block join gradient");
}

template <class T>
int launch_join_grad(JoinGradParams& p, bool vec, cudaStream_t stream) {
  const int nv = row_frags(p.cols);
  p.stage_bytes = 0;
  for (int which = 0; which < 4; ++which) {
    const bool packed = (which == kInY && p.y8.codes) || (which == kInH && p.h8.codes);
    p.frag_at[which] = p.stage_bytes;
    p.frag_bytes[which] = packed ? 8 : 8 * sizeof(T);
    if (which == kInDh || which == kInY || p.du.data)
      p.stage_bytes += p.frag_bytes[which] * nv * p.tpr;
  }
  // the vector form needs room for at least one row of the ring
  vec = vec && p.tpr * 16 * nv * sizeof(float) + p.stage_bytes <= kJoinSmem / ctas_per_sm(p.cols);
  switch (nv) {
    case 1:
      return vec ? launch_join_grad_at<T, true, 1>(p, stream)
                 : launch_join_grad_at<T, false, 1>(p, stream);
    case 2:
      return vec ? launch_join_grad_at<T, true, 2>(p, stream)
                 : launch_join_grad_at<T, false, 2>(p, stream);
    default:
      return vec ? launch_join_grad_at<T, true, 4>(p, stream)
                 : launch_join_grad_at<T, false, 4>(p, stream);
  }
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
  auto one = [&](const char* name, const void* q, int64_t len, int64_t size, bool w) {
    return q ? take_matrix(name, dpopt_matrix{const_cast<void*>(q), len}, 1, len, size, w, &dummy,
                           s, &n)
             : DPOPT_OK;
  };
  DPOPT_TRY(one("w_post", a->w_post, cols, ps, false));
  DPOPT_TRY(one("w_pre", a->w_pre, cols, ps, false));
  DPOPT_TRY(one("rstd_post", a->rstd_post, rows, 4, true));
  DPOPT_TRY(one("rstd_pre", a->rstd_pre, rows, 4, true));
  if (a->y8.codes) DPOPT_TRY(take_act8("y8", a->y8, rows, cols, true, &p.y8, s, &n));
  if (a->h8.codes) DPOPT_TRY(take_act8("h8", a->h8, rows, cols, true, &p.h8, s, &n));
  if (a->u8.codes) DPOPT_TRY(take_act8("u8", a->u8, rows, cols, true, &p.u8, s, &n));
  DPOPT_TRY(check_overlaps(s, n));
  p.rows = rows;
  p.cols = (int)cols;
  p.tpr = row_threads(cols);
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
  const bool vec = cols % 8 == 0 && vec_ok(p.h) && vec_ok(p.y) && vec_ok(p.h_out) &&
                   vec_ok(p.u) && vec_ok(p.y8) && vec_ok(p.h8) && vec_ok(p.u8);
  const cudaStream_t st = (cudaStream_t)stream;
  if (a->dtype == DPOPT_GRAD_BF16) return launch_join<bf16>(p, vec, st);
  if (a->dtype == DPOPT_GRAD_F16) return launch_join<fp16>(p, vec, st);
  return launch_join<float>(p, vec, st);
}

int dpopt_block_join_scratch_bytes(int64_t rows, int64_t cols, int64_t gate_rows,
                                   int64_t* bytes_out) {
  if (!bytes_out || rows < 0 || cols < 0 || gate_rows < 0)
    return fail(DPOPT_ERR_INVALID_ARG, "block join scratch: null output or a negative size");
  if (cols > DPOPT_JOIN_MAX_COLS)
    return fail(DPOPT_ERR_UNSUPPORTED, "cols %lld exceeds %d", (long long)cols,
                DPOPT_JOIN_MAX_COLS);
  *bytes_out = part_count(rows, cols) * kPartSlots * whole_blocks(cols) *
               (int64_t)sizeof(float);
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
  auto one = [&](const char* name, const void* q, int64_t len, int64_t size, bool w) {
    return q ? take_matrix(name, dpopt_matrix{const_cast<void*>(q), len}, 1, len, size, w, &dummy,
                           s, &n)
             : DPOPT_OK;
  };
  DPOPT_TRY(one("w_post", a->w_post, cols, ps, false));
  DPOPT_TRY(one("w_pre", a->w_pre, cols, ps, false));
  DPOPT_TRY(one("rstd_post", a->rstd_post, rows, 4, false));
  DPOPT_TRY(one("rstd_pre", a->rstd_pre, rows, 4, false));
  DPOPT_TRY(one("dw_post", a->dw_post, cols, ps, true));
  DPOPT_TRY(one("dw_pre", a->dw_pre, cols, ps, true));
  int64_t need = 0;
  DPOPT_TRY(dpopt_block_join_scratch_bytes(rows, cols, a->gate_rows, &need));
  if (need > 0) {
    if (!a->scratch || (uintptr_t)a->scratch % 256)
      return fail(DPOPT_ERR_INVALID_ARG, "scratch must be non-null and 256-byte aligned");
    if (a->scratch_bytes < need)
      return fail(DPOPT_ERR_INVALID_ARG, "scratch holds %lld bytes, %lld are needed",
                  (long long)a->scratch_bytes, (long long)need);
    DPOPT_TRY(one("scratch", a->scratch, need, 1, true));
  }
  DPOPT_TRY(check_overlaps(s, n));
  p.rows = rows;
  p.cols = (int)cols;
  p.tpr = row_threads(cols);
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
  const int64_t parts = part_count(rows, cols);
  p.width = (int)whole_blocks(cols);
  p.per = part_rows(rows, cols);
  p.parts = parts;
  if (rows > 0) {
    const bool vec = cols % 8 == 0 && vec_ok(p.dh_out) && vec_ok(p.du) && vec_ok(p.y) &&
                     vec_ok(p.h_out) && vec_ok(p.dh) && vec_ok(p.dy) && vec_ok(p.y8) &&
                     vec_ok(p.h8);
    const cudaStream_t st = (cudaStream_t)stream;
    DPOPT_TRY(a->dtype == DPOPT_GRAD_BF16  ? launch_join_grad<bf16>(p, vec, st)
              : a->dtype == DPOPT_GRAD_F16 ? launch_join_grad<fp16>(p, vec, st)
                                           : launch_join_grad<float>(p, vec, st));
  }
  if (!p.dw_pre && !p.dw_post && !p.dgate.data) return DPOPT_OK;
  // gate rows that cross a part's border: one for all rows, or at most one per
  // border (none when the parts are whole numbers of gate rows)
  unsigned gate_sums = 0;
  if (p.dgate.data) {
    if (a->gate_rows == 0)
      gate_sums = rows == 0 || parts > 1;
    else if (rows > 0 && part_rows(rows, cols) % a->gate_rows != 0)
      gate_sums = (unsigned)(parts - 1);
  }
  if (!p.dw_pre && !p.dw_post && gate_sums == 0) return DPOPT_OK;
  const dim3 grid((unsigned)((cols + 31) / 32), 2 + gate_sums);
  return launched(launch_pdl(block_join_finish_kernel, grid, dim3(32 * kFinishRuns), 0,
                             (cudaStream_t)stream, p),
                  "block join gradient sums");
}

}  // extern "C"
