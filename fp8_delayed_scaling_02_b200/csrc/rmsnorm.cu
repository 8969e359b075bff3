// fp8_rmsnorm / fp8_rmsnorm_backward: the norm that feeds an FP8 linear, with
// the residual's addition before it and the FP8 cast behind it, and its
// gradient (sm_100a).
//
// Both are streams bound by HBM: forward 2 reads, 1 write and 1 code byte per
// element with a residual, backward 3 reads and 1 write.  So each element is
// read once and stays in registers, packed as it lies in memory:
//   * a group of W warps (1, 2, 4, 8 or 16) owns a row, each thread V <= 4
//     vectors of 8 elements at fixed columns; gamma for those columns is read
//     once per thread and kept, and so are the partial sums of dgamma;
//   * the row's statistics cross lanes by shuffles and, where W > 1, warps by
//     one shared word each and a named barrier of the group alone;
//   * groups walk over the rows of one wave of resident blocks;
//   * dgamma: each block adds its groups' partial sums in order and writes one
//     float32 row; a second launch adds those rows, in order, so every bit
//     depends on the sizes and the device only.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "amax_fold.cuh"
#include "colsum.cuh"
#include "common.cuh"
#include "elem_io.cuh"
#include "fp8_ring.cuh"
#include "fp8ds_layer.h"
#include "host_util.cuh"
#include "row_vec.cuh"

namespace fp8ds {
namespace {

constexpr int kMaxCols = 16384;  // 16 warps x 32 lanes x 4 vectors x 8
constexpr int kMaxVec = 4;

struct NormArgs {
  const uint8_t* x;
  const uint8_t* res;
  const void* gamma;
  int gamma_f32;
  float eps;
  int64_t rows;
  int cols;
  int log_w;         // warps per row, log2
  uint8_t* h;
  uint8_t* y;
  float* rstd;
  uint8_t* codes;
  int fmt;
  int fold;          // the codes' scale is the ring's, which the last block folds
  float* row_sinv;   // or every row has its own
  RingArgs ring;
};

struct NormBwdArgs {
  const uint8_t* dy;
  const uint8_t* h;
  const uint8_t* dres;
  const float* rstd;
  const void* gamma;
  int gamma_f32;
  int64_t rows;
  int cols;
  int log_w;
  uint8_t* dx;
  float* partial;    // [gridDim.x][cols] sums of dy * n, or null
};

// Sums (or maxima) over the threads of one row's group.  Every thread of the
// group calls it; the result is the same in all of them.  The two halves of
// `sm` alternate between calls: a warp can write a half again only after a
// barrier that every reader of its last contents has reached.
template <int NT>
struct GroupReduce {
  float* sm;  // [2][NT / 32]
  int warps, group, warp_in_group, flip;

  template <typename Op>
  __device__ __forceinline__ float run(float v, Op op) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (warps == 1) return v;
    float* buf = sm + flip * (NT / 32) + group * warps;
    if ((threadIdx.x & 31) == 0) buf[warp_in_group] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * warps) : "memory");
    float r = buf[0];
    for (int w = 1; w < warps; ++w) r = op(r, buf[w]);
    flip ^= 1;
    return r;
  }
  __device__ __forceinline__ float sum(float v) {
    return run(v, [](float a, float b) { return a + b; });
  }
  __device__ __forceinline__ float max(float v) {
    return run(v, [](float a, float b) { return fmaxf(a, b); });
  }
};

template <int DT>
__device__ __forceinline__ void load_gamma8(const void* gamma, int f32, int c, int cols, float (&g)[8]) {
  const uint8_t* p = static_cast<const uint8_t*>(gamma);
  if (f32) unpack8<FP8_IN_FP32>(load8<FP8_IN_FP32, false>(p, c, cols), g);
  else unpack8<DT>(load8<DT, false>(p, c, cols), g);
}

template <int DT, bool kAligned, int V, int NT>
__global__ void __launch_bounds__(NT) rmsnorm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kB = In<DT>::kBytes;
  __shared__ float red[2 * (NT / 32)];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int warps = 1 << a.log_w;
  const int warp = threadIdx.x >> 5;
  const int group = warp >> a.log_w;
  const int groups = (NT / 32) >> a.log_w;
  const int t = threadIdx.x - ((group << a.log_w) << 5);
  const int stride = 256 << a.log_w;  // columns between a thread's vectors
  GroupReduce<NT> gr{red, warps, group, warp - (group << a.log_w), 0};

  const bool ring_mode = a.fold != 0;
  const float s_ring = ring_mode ? *a.ring.scale : 1.0f;
  RingCache rc{0.0f, 0};
  if (ring_mode) rc = prefetch_ring(a.ring);
  float gm[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) load_gamma8<DT>(a.gamma, a.gamma_f32, 8 * t + v * stride, a.cols, gm[v]);

  const float inv_cols = __frcp_rn(float(a.cols));
  const float fmax = a.fmt == FP8_E5M2 ? kE5M2Max : kE4M3Max;
  float amax = 0.0f;
  for (int64_t row = int64_t(blockIdx.x) * groups + group; row < a.rows; row += int64_t(gridDim.x) * groups) {
    const int64_t off = row * a.cols * kB;
    Vec8<DT> h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = load8<DT, kAligned>(a.x + off, 8 * t + v * stride, a.cols);
    if (a.res != nullptr) {
      Vec8<DT> r[V];
#pragma unroll
      for (int v = 0; v < V; ++v) r[v] = load8<DT, kAligned>(a.res + off, 8 * t + v * stride, a.cols);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float p[8], q[8];
        unpack8<DT>(h[v], p);
        unpack8<DT>(r[v], q);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] += q[i];
        h[v] = pack8<DT>(p);
        store8<DT, kAligned>(a.h + off, 8 * t + v * stride, a.cols, h[v]);
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float p[8];
      unpack8<DT>(h[v], p);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(p[i], p[i], ss);
    }
    const float rstd = rsqrtf(fmaf(gr.sum(ss), inv_cols, a.eps));
    if (a.rstd != nullptr && t == 0) a.rstd[row] = rstd;
    float s = s_ring;
    if (a.row_sinv != nullptr) {
      float m = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float p[8];
        unpack8<DT>(h[v], p);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(__fmul_rn(__fmul_rn(p[i], rstd), gm[v][i])));
      }
      m = gr.max(m);
      s = 1.0f;
      if (m > 0.0f && isfinite(m)) {
        const float q = __fdiv_rn(fmax, m);
        if (isfinite(q) && q > 0.0f) s = q;
      }
      if (t == 0) a.row_sinv[row] = __frcp_rn(s);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * t + v * stride;
      float p[8];
      unpack8<DT>(h[v], p);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = __fmul_rn(__fmul_rn(p[i], rstd), gm[v][i]);
        amax = fmaxf(amax, fabsf(p[i]));  // 0 beyond the row's end
      }
      if (a.y != nullptr) store8<DT, kAligned>(a.y + off, c, a.cols, pack8<DT>(p));
      if (a.codes != nullptr) {
        uint32_t lo, hi;
        if (a.fmt == FP8_E5M2) {
          lo = cvt4<FP8_E5M2>(p[0], p[1], p[2], p[3], s);
          hi = cvt4<FP8_E5M2>(p[4], p[5], p[6], p[7], s);
        } else {
          lo = cvt4<FP8_E4M3>(p[0], p[1], p[2], p[3], s);
          hi = cvt4<FP8_E4M3>(p[4], p[5], p[6], p[7], s);
        }
        store8_codes<kAligned>(a.codes + row * a.cols, c, a.cols, lo, hi);
      }
    }
  }
  if (ring_mode) {
    if (a.fmt == FP8_E5M2) amax_ticket_fold<FP8_E5M2, NT>(amax, a.ring, s_ring, rc, gridDim.x);
    else amax_ticket_fold<FP8_E4M3, NT>(amax, a.ring, s_ring, rc, gridDim.x);
  }
}

template <int DT, bool kAligned, int V, int NT>
__global__ void __launch_bounds__(NT) rmsnorm_bwd_kernel(const __grid_constant__ NormBwdArgs a) {
  constexpr int kB = In<DT>::kBytes;
  // Rows of up to 1024 V columns (four warps or fewer) share a block with
  // other groups, whose dgamma sums are added here.
  __shared__ float red[2 * (NT / 32)];
  __shared__ float sum_s[NT == 256 ? 1024 * V : 1];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int warps = 1 << a.log_w;
  const int warp = threadIdx.x >> 5;
  const int group = warp >> a.log_w;
  const int groups = (NT / 32) >> a.log_w;
  const int t = threadIdx.x - ((group << a.log_w) << 5);
  const int stride = 256 << a.log_w;
  GroupReduce<NT> gr{red, warps, group, warp - (group << a.log_w), 0};
  float gm[V][8], dg[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    load_gamma8<DT>(a.gamma, a.gamma_f32, 8 * t + v * stride, a.cols, gm[v]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[v][i] = 0.0f;
  }
  const float inv_cols = __frcp_rn(float(a.cols));
  for (int64_t row = int64_t(blockIdx.x) * groups + group; row < a.rows; row += int64_t(gridDim.x) * groups) {
    const int64_t off = row * a.cols * kB;
    const float rstd = a.rstd[row];
    Vec8<DT> dy[V], h[V], dr[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      dy[v] = load8<DT, kAligned>(a.dy + off, 8 * t + v * stride, a.cols);
      h[v] = load8<DT, kAligned>(a.h + off, 8 * t + v * stride, a.cols);
      if (a.dres != nullptr) dr[v] = load8<DT, kAligned>(a.dres + off, 8 * t + v * stride, a.cols);
    }
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float d[8], n[8];
      unpack8<DT>(dy[v], d);
      unpack8<DT>(h[v], n);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = d[i] * (n[i] * rstd);
        dg[v][i] += e;
        dot = fmaf(e, gm[v][i], dot);
      }
    }
    const float c1 = gr.sum(dot) * inv_cols;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float d[8], n[8], e[8];
      unpack8<DT>(dy[v], d);
      unpack8<DT>(h[v], n);
      if (a.dres != nullptr) {
        unpack8<DT>(dr[v], e);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = fmaf(rstd, fmaf(-(n[i] * rstd), c1, d[i] * gm[v][i]), e[i]);
      store8<DT, kAligned>(a.dx + off, 8 * t + v * stride, a.cols, pack8<DT>(e));
    }
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + int64_t(blockIdx.x) * a.cols;
  if (groups > 1) {
    for (int g = 0; g < groups; ++g) {
      if (group == g) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = 8 * t + v * stride;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (g > 0) dg[v][i] += sum_s[c + i];
            sum_s[c + i] = dg[v][i];
          }
        }
      }
      __syncthreads();
    }
    if (group != groups - 1) return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * t + v * stride;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < a.cols) out[c + i] = dg[v][i];
  }
}

// ---- host side -----------------------------------------------------------------

// How a row is split: W = 2^log_w warps and V vectors per thread.
struct RowSplit {
  int log_w, v, nt;
};

RowSplit split_row(int64_t rows, int64_t cols) {
  const int64_t vecs = (cols + 7) / 8;
  RowSplit s{0, 1, 256};
  while ((vecs + (32 << s.log_w) - 1) / (32 << s.log_w) > kMaxVec) ++s.log_w;
  // Few rows: more warps on each, so that a row's loads are in flight at once.
  while (s.log_w < 3 && vecs > (32 << s.log_w) && (rows << s.log_w) < 148 * 8) ++s.log_w;
  s.v = int((vecs + (32 << s.log_w) - 1) / (32 << s.log_w));
  s.nt = s.log_w > 3 ? 512 : 256;
  return s;
}

int64_t bwd_blocks(int64_t rows, int64_t cols, int sms) {
  const RowSplit s = split_row(rows, cols);
  const int64_t groups = (s.nt / 32) >> s.log_w;
  return std::max<int64_t>(1, std::min<int64_t>((rows + groups - 1) / groups, 2 * int64_t(sms)));
}

int norm_shape_check(int dtype, int64_t rows, int64_t cols) {
  if (dtype < FP8_IN_BF16 || dtype > FP8_IN_FP32) return FP8_ERR_INVALID_ARG;
  if (rows < 0 || cols < 1) return FP8_ERR_INVALID_ARG;
  if (cols > kMaxCols || rows > INT32_MAX) return FP8_ERR_UNSUPPORTED;
  return FP8_OK;
}

template <typename K, typename A>
int launch_rows(K kern, const A& a, int64_t rows, const RowSplit& s, int64_t most, int (&cached)[64],
                cudaStream_t st) {
  const int bps = resident_blocks(kern, s.nt, cached);
  const int sms = sm_count_current();
  if (bps < 1 || sms < 1) return FP8_ERR_CUDA;
  const int64_t groups = (s.nt / 32) >> s.log_w;
  int64_t grid = std::max<int64_t>(1, std::min<int64_t>((rows + groups - 1) / groups, int64_t(sms) * bps));
  if (most > 0) grid = most;
  return launch_pdl(kern, dim3(unsigned(grid)), dim3(s.nt), 0, st, 1, a) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

template <int DT, bool kAligned, int V, int NT>
int launch_fwd1(const NormArgs& a, const RowSplit& s, cudaStream_t st) {
  static int cached[64] = {0};
  return launch_rows(rmsnorm_kernel<DT, kAligned, V, NT>, a, a.rows, s, 0, cached, st);
}

template <int DT, bool kAligned>
int launch_fwd(const NormArgs& a, const RowSplit& s, cudaStream_t st) {
  if (s.nt == 512) return s.v <= 3 ? launch_fwd1<DT, kAligned, 3, 512>(a, s, st) : launch_fwd1<DT, kAligned, 4, 512>(a, s, st);
  switch (s.v) {
    case 1: return launch_fwd1<DT, kAligned, 1, 256>(a, s, st);
    case 2: return launch_fwd1<DT, kAligned, 2, 256>(a, s, st);
    case 3: return launch_fwd1<DT, kAligned, 3, 256>(a, s, st);
    default: return launch_fwd1<DT, kAligned, 4, 256>(a, s, st);
  }
}

template <int DT, bool kAligned, int V, int NT>
int launch_bwd1(const NormBwdArgs& a, const RowSplit& s, int64_t grid, cudaStream_t st) {
  static int cached[64] = {0};
  return launch_rows(rmsnorm_bwd_kernel<DT, kAligned, V, NT>, a, a.rows, s, grid, cached, st);
}

template <int DT, bool kAligned>
int launch_bwd(const NormBwdArgs& a, const RowSplit& s, int64_t g, cudaStream_t st) {
  if (s.nt == 512) return s.v <= 3 ? launch_bwd1<DT, kAligned, 3, 512>(a, s, g, st) : launch_bwd1<DT, kAligned, 4, 512>(a, s, g, st);
  switch (s.v) {
    case 1: return launch_bwd1<DT, kAligned, 1, 256>(a, s, g, st);
    case 2: return launch_bwd1<DT, kAligned, 2, 256>(a, s, g, st);
    case 3: return launch_bwd1<DT, kAligned, 3, 256>(a, s, g, st);
    default: return launch_bwd1<DT, kAligned, 4, 256>(a, s, g, st);
  }
}

}  // namespace
}  // namespace fp8ds

using namespace fp8ds;

extern "C" int fp8_rmsnorm(const fp8_rmsnorm_args* p, fp8_stream_t stream) {
  if (p == nullptr) return FP8_ERR_INVALID_ARG;
  int rc = norm_shape_check(p->dtype, p->rows, p->cols);
  if (rc == FP8_ERR_INVALID_ARG) return rc;
  if (!(p->eps > 0.0f) || p->eps > 3.0e38f) return FP8_ERR_INVALID_ARG;
  if (p->gamma == nullptr || (p->rows > 0 && p->x == nullptr)) return FP8_ERR_INVALID_ARG;
  if (p->rows > 0 && (p->residual == nullptr) != (p->h == nullptr)) return FP8_ERR_INVALID_ARG;
  const bool ring_mode = p->ring.scale != nullptr || p->amax_out != nullptr;
  if (p->rows > 0 && p->codes == nullptr && p->y == nullptr) return FP8_ERR_INVALID_ARG;
  if (p->codes == nullptr && p->rows > 0 && (ring_mode || p->row_sinv != nullptr)) return FP8_ERR_INVALID_ARG;
  if (p->codes != nullptr || ring_mode || p->row_sinv != nullptr) {
    if (p->fmt != FP8_E4M3 && p->fmt != FP8_E5M2) return FP8_ERR_INVALID_ARG;
    const fp8_ring& r = p->ring;
    if (p->row_sinv != nullptr) {
      if (ring_mode) return FP8_ERR_INVALID_ARG;
    } else if (!r.scale || !r.scale_inv || !r.scratch || (p->amax_out == nullptr && (!r.history || !r.idx))) {
      return FP8_ERR_INVALID_ARG;
    }
    if (p->row_sinv == nullptr && !on(r.scratch, 8)) return FP8_ERR_UNSUPPORTED;
  }
  if (rc != FP8_OK) return rc;
  const int eb = p->dtype == FP8_IN_FP32 ? 4 : 2;
  if (!on(p->x, eb) || !on(p->residual, eb) || !on(p->h, eb) || !on(p->y, eb) || !on(p->gamma, p->gamma_f32 ? 4 : eb) ||
      !on(p->rstd, 4) || !on(p->row_sinv, 4))
    return FP8_ERR_UNSUPPORTED;
  const size_t n = size_t(p->rows) * size_t(p->cols);
  const Span spans[] = {{p->x, n * eb, false, false, true},
                        {p->residual, n * eb, false, false, true},
                        {p->gamma, size_t(p->cols) * (p->gamma_f32 ? 4 : eb), false, false, false},
                        {p->h, n * eb, true, true, false},
                        {p->y, n * eb, true, true, false},
                        {p->rstd, size_t(p->rows) * 4, true, false, false},
                        {p->codes, n, true, false, false},
                        {p->row_sinv, size_t(p->rows) * 4, true, false, false}};
  if (spans_clash(spans, 8)) return FP8_ERR_INVALID_ARG;
  if (p->rows == 0 && !ring_mode) return FP8_OK;
  NormArgs a{};
  a.x = static_cast<const uint8_t*>(p->x);
  a.res = static_cast<const uint8_t*>(p->residual);
  a.gamma = p->gamma;
  a.gamma_f32 = p->gamma_f32 != 0 || p->dtype == FP8_IN_FP32;
  a.eps = p->eps;
  a.rows = p->rows;
  a.cols = int(p->cols);
  a.h = static_cast<uint8_t*>(p->h);
  a.y = static_cast<uint8_t*>(p->y);
  a.rstd = p->rstd;
  a.codes = p->codes;
  a.fold = ring_mode;
  a.fmt = p->fmt;
  a.row_sinv = p->row_sinv;
  if (ring_mode)
    a.ring = RingArgs{p->ring.history, p->ring.idx, p->ring.scale, p->ring.scale_inv, p->ring.scratch, p->amax_out};
  const RowSplit s = split_row(p->rows, p->cols);
  a.log_w = s.log_w;
  const bool al = p->cols % 8 == 0 && on(p->x, 16) && on(p->residual, 16) && on(p->h, 16) && on(p->y, 16) &&
                  on(p->codes, 8);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (p->dtype) {
    case FP8_IN_BF16: return al ? launch_fwd<FP8_IN_BF16, true>(a, s, st) : launch_fwd<FP8_IN_BF16, false>(a, s, st);
    case FP8_IN_FP16: return al ? launch_fwd<FP8_IN_FP16, true>(a, s, st) : launch_fwd<FP8_IN_FP16, false>(a, s, st);
    default: return al ? launch_fwd<FP8_IN_FP32, true>(a, s, st) : launch_fwd<FP8_IN_FP32, false>(a, s, st);
  }
}

extern "C" size_t fp8_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || cols > kMaxCols || rows > INT32_MAX) return 0;
  const int sms = sm_count_current();
  if (sms <= 0) return 0;
  const int64_t n = bwd_blocks(rows, cols, sms);
  return n > 1 ? size_t(n) * size_t(cols) * 4 : 0;
}

extern "C" int fp8_rmsnorm_backward(const fp8_rmsnorm_backward_args* p, fp8_stream_t stream) {
  if (p == nullptr) return FP8_ERR_INVALID_ARG;
  const int rc = norm_shape_check(p->dtype, p->rows, p->cols);
  if (rc == FP8_ERR_INVALID_ARG) return rc;
  if (p->rows > 0 && (p->dy == nullptr || p->h == nullptr || p->rstd == nullptr || p->gamma == nullptr ||
                      p->dx == nullptr))
    return FP8_ERR_INVALID_ARG;
  if (rc != FP8_OK) return rc;
  const int eb = p->dtype == FP8_IN_FP32 ? 4 : 2;
  if (!on(p->dy, eb) || !on(p->h, eb) || !on(p->dres, eb) || !on(p->dx, eb) || !on(p->gamma, p->gamma_f32 ? 4 : eb) ||
      !on(p->rstd, 4) || !on(p->dgamma, 4) || !on(p->workspace, 4))
    return FP8_ERR_UNSUPPORTED;
  const size_t n = size_t(p->rows) * size_t(p->cols);
  const Span spans[] = {{p->dy, n * eb, false, false, true},
                        {p->h, n * eb, false, false, false},
                        {p->dres, n * eb, false, false, true},
                        {p->rstd, size_t(p->rows) * 4, false, false, false},
                        {p->gamma, size_t(p->cols) * (p->gamma_f32 ? 4 : eb), false, false, false},
                        {p->dx, n * eb, true, true, false},
                        {p->dgamma, size_t(p->cols) * 4, true, false, false},
                        {p->workspace, p->dgamma ? p->workspace_bytes : 0, true, false, false}};
  if (spans_clash(spans, 8)) return FP8_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p->rows == 0 && p->dgamma == nullptr) return FP8_OK;
  const int sms = sm_count_current();
  if (sms <= 0) return FP8_ERR_CUDA;
  const RowSplit s = split_row(p->rows, p->cols);
  const int64_t grid = bwd_blocks(p->rows, p->cols, sms);
  NormBwdArgs a{};
  a.dy = static_cast<const uint8_t*>(p->dy);
  a.h = static_cast<const uint8_t*>(p->h);
  a.dres = static_cast<const uint8_t*>(p->dres);
  a.rstd = p->rstd;
  a.gamma = p->gamma;
  a.gamma_f32 = p->gamma_f32 != 0 || p->dtype == FP8_IN_FP32;
  a.rows = p->rows;
  a.cols = int(p->cols);
  a.log_w = s.log_w;
  a.dx = static_cast<uint8_t*>(p->dx);
  if (p->rows == 0) {  // no rows: the empty sum
    return launch_colsum(nullptr, 0, p->cols, p->dgamma, st);
  }
  if (p->dgamma != nullptr) {
    if (grid > 1) {
      if (p->workspace == nullptr || p->workspace_bytes < size_t(grid) * size_t(p->cols) * 4) return FP8_ERR_INVALID_ARG;
      a.partial = static_cast<float*>(p->workspace);
    } else {
      a.partial = p->dgamma;  // one block: its sums are the result
    }
  }
  const bool al = p->cols % 8 == 0 && on(p->dy, 16) && on(p->h, 16) && on(p->dres, 16) && on(p->dx, 16);
  int r;
  switch (p->dtype) {
    case FP8_IN_BF16: r = al ? launch_bwd<FP8_IN_BF16, true>(a, s, grid, st) : launch_bwd<FP8_IN_BF16, false>(a, s, grid, st); break;
    case FP8_IN_FP16: r = al ? launch_bwd<FP8_IN_FP16, true>(a, s, grid, st) : launch_bwd<FP8_IN_FP16, false>(a, s, grid, st); break;
    default: r = al ? launch_bwd<FP8_IN_FP32, true>(a, s, grid, st) : launch_bwd<FP8_IN_FP32, false>(a, s, grid, st); break;
  }
  if (r != FP8_OK || p->dgamma == nullptr || grid == 1) return r;
  return launch_colsum(a.partial, int(grid), p->cols, p->dgamma, st);
}
