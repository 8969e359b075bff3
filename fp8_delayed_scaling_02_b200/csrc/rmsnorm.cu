// fp8_rmsnorm / fp8_rmsnorm_backward: the norm that feeds an FP8 linear, with
// the residual's addition before it and the FP8 cast behind it, and its
// gradient (sm_100a).
//
// Both are streams: forward 2 reads, 1 write and 1 code byte per element with a
// residual, backward 3 reads and 1 write.  So each element is read once, packed as
// it lies in memory, and stays with its thread:
//   * a group of W warps owns a row, each thread V vectors of 8 elements at
//     fixed columns (1536 columns: forward W = 3, V = 2, backward W = 6, V = 1, no
//     idle lanes); the next row's loads go out before the row in work is reduced,
//     as far as the registers last;
//   * the row's statistics cross lanes by shuffles and, where W > 1, warps by
//     one shared word each and a named barrier of the group alone;
//   * gamma comes from L1 for each row, its load ahead of the reduction: kept
//     in registers it costs the occupancy that keeps the loads in flight (the
//     forward with four vectors, which loads no row ahead, keeps it);
//   * groups walk over the rows of one wave of resident blocks;
//   * dgamma: partial sums per thread, then each block adds its groups' in
//     order and writes one float32 row; a second launch adds those rows, in
//     order, so every bit depends on the sizes, the type and the device only.
// At 8192 x 1536 bf16 both are as near to their issue slots (64%) as to HBM: 16.4
// us forward, 23.0 backward (13.5 and 15.4 at the copy rate).  Rows above 8192
// columns do not fit the registers in the gradient (176 to 400 bytes of spills a
// thread with four vectors; 2048 x 12288 float32 123 us, 61.6 at the copy rate), nor
// in the forward of float32 (384 bytes, unaligned 996; 74.9 us, 50.0).  Rows that
// are no multiple of 8 elements or start off the 16-byte grid pay for loads that
// cover the neighbour's granule and stores in pieces: 8192 x 1537 39.3 and 61.3 us.
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
constexpr int kMaxWarps = 16;    // per row
constexpr int kRedWords = 24;    // warps of a block, at most

struct NormArgs {
  const uint8_t* x;
  const uint8_t* res;
  const void* gamma;
  int gamma_f32;
  float eps;
  int64_t rows;
  int cols;
  int warps, groups; // warps per row, rows in work per block
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
  int warps, groups;
  uint8_t* dx;
  float* partial;    // [gridDim.x][cols] sums of dy * n, or null
};

// Sums (or maxima) over the threads of one row's group.  Every thread of the
// group calls it; the result is the same in all of them.  The two halves of
// `sm` alternate between calls: a warp can write a half again only after a
// barrier that every reader of its last contents has reached.
struct GroupReduce {
  float* sm;  // [2][kRedWords]
  int warps, group, warp_in_group, flip;

  template <typename Op>
  __device__ __forceinline__ float run(float v, Op op) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (warps == 1) return v;
    float* buf = sm + flip * kRedWords + group * warps;
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

// Eight values of gamma (kAligned: gamma too is 16-byte aligned).
template <int DT, bool kAligned>
__device__ __forceinline__ void load_gamma8(const void* gamma, int f32, int c, int cols, float (&g)[8]) {
  const uint8_t* p = static_cast<const uint8_t*>(gamma);
  if (f32) unpack8<FP8_IN_FP32>(load8<FP8_IN_FP32, kAligned>(p, c, cols), g);
  else unpack8<DT>(load8<DT, kAligned>(p, c, cols), g);
}

// Blocks per SM that the forward's registers allow, for the loads in flight.  Two
// 16-bit vectors per thread, 8192 x 1536 in blocks of three, four and (126
// registers) two: 16.6, 19.1 and 21.7 us; 8192 x 1537: 43.9, 38.9 (with 48 bytes of
// spills a thread) and 56.2.
template <int DT, bool kAligned, int V, int NT>
constexpr int kFwdBlocks = NT > 256 ? 1 : V == 1 ? 4 : In<DT>::kBytes == 4 ? 2 : kAligned ? 3 : 4;

template <int DT, bool kAligned, int V, int NT>
__global__ void __launch_bounds__(NT, (kFwdBlocks<DT, kAligned, V, NT>)) rmsnorm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kB = In<DT>::kBytes;
  // Up to two vectors per thread: the next row's loads go out ahead of the row
  // in work, and gamma is read again for each row.  Four: gamma is kept instead.
  constexpr bool kAhead = V <= 2;
  __shared__ float red[2 * kRedWords];
  __shared__ float hist_s[kHistoryLen];
  __shared__ int idx_s;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / a.warps;
  const int t = threadIdx.x - group * a.warps * 32;
  const int stride = 256 * a.warps;  // columns between a thread's vectors
  GroupReduce gr{red, a.warps, group, warp - group * a.warps, 0};

  const float s_ring = a.fold ? *a.ring.scale : 1.0f;
  if (a.fold && a.ring.amax_out == nullptr) {  // not written before the last block's fold
    if (threadIdx.x < kHistoryLen) hist_s[threadIdx.x] = a.ring.history[threadIdx.x];
    if (threadIdx.x == kHistoryLen) idx_s = *a.ring.idx;
  }
  const float inv_cols = __frcp_rn(float(a.cols));
  const float fmax = a.fmt == FP8_E5M2 ? kE5M2Max : kE4M3Max;
  const int64_t step = int64_t(gridDim.x) * a.groups;
  float amax = 0.0f;
  Vec8<DT> nx[V], nr[V];  // the next row of x and residual
  auto load = [&](int64_t row) {
    const int64_t off = row * a.cols * kB;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      nx[v] = load8<DT, kAligned>(a.x + off, 8 * t + v * stride, a.cols);
      if (a.res != nullptr) nr[v] = load8<DT, kAligned>(a.res + off, 8 * t + v * stride, a.cols);
    }
  };
  float gm[V][8];
  auto load_gamma = [&]() {
#pragma unroll
    for (int v = 0; v < V; ++v) load_gamma8<DT, kAligned>(a.gamma, a.gamma_f32, 8 * t + v * stride, a.cols, gm[v]);
  };
  if (!kAhead) load_gamma();
  int64_t row = int64_t(blockIdx.x) * a.groups + group;
  if (row < a.rows) load(row);
  for (; row < a.rows; row += step) {
    const int64_t off = row * a.cols * kB;
    float p[V][8];  // h, then v
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      unpack8<DT>(nx[v], p[v]);
      if (a.res != nullptr) {
        float q[8];
        unpack8<DT>(nr[v], q);
#pragma unroll
        for (int i = 0; i < 8; i += 2) add2(p[v][i], p[v][i + 1], q[i], q[i + 1]);
        unpack8<DT>(pack8<DT>(p[v]), p[v]);
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float x = p[v][i], y = p[v][i + 1];
        fma2v(x, y, x, y, s0, s1);
        s0 = x, s1 = y;
      }
    }
    if (kAhead && row + step < a.rows) load(row + step);
    if (a.res != nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v) store8<DT, kAligned>(a.h + off, 8 * t + v * stride, a.cols, pack8<DT>(p[v]));
    }
    if (kAhead) load_gamma();
    const float rstd = rsqrtf(fmaf(gr.sum(s0 + s1), inv_cols, a.eps));
    if (a.rstd != nullptr && t == 0) a.rstd[row] = rstd;
    float m = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        scale2(p[v][i], p[v][i + 1], rstd);
        mul2(p[v][i], p[v][i + 1], gm[v][i], gm[v][i + 1]);
        m = fmaxf(m, fmaxf(fabsf(p[v][i]), fabsf(p[v][i + 1])));  // 0 beyond the row's end
      }
    amax = fmaxf(amax, m);
    float s = s_ring;
    if (a.row_sinv != nullptr) {
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
      if (a.y != nullptr) store8<DT, kAligned>(a.y + off, c, a.cols, pack8<DT>(p[v]));
      if (a.codes != nullptr) {
        uint32_t lo, hi;
        if (a.fmt == FP8_E5M2) {
          lo = cvt4<FP8_E5M2>(p[v][0], p[v][1], p[v][2], p[v][3], s);
          hi = cvt4<FP8_E5M2>(p[v][4], p[v][5], p[v][6], p[v][7], s);
        } else {
          lo = cvt4<FP8_E4M3>(p[v][0], p[v][1], p[v][2], p[v][3], s);
          hi = cvt4<FP8_E4M3>(p[v][4], p[v][5], p[v][6], p[v][7], s);
        }
        store8_codes<kAligned>(a.codes + row * a.cols, c, a.cols, lo, hi);
      }
    }
    if (!kAhead && row + step < a.rows) load(row + step);
  }
  if (!a.fold) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  __syncthreads();  // every group is done with `red`
  if (lane == 0) red[warp] = amax;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < a.warps * a.groups; ++w) amax = fmaxf(amax, red[w]);
  if (a.fmt == FP8_E5M2) commit_block_amax<FP8_E5M2>(amax, a.ring, s_ring, hist_s, idx_s, gridDim.x);
  else commit_block_amax<FP8_E4M3>(amax, a.ring, s_ring, hist_s, idx_s, gridDim.x);
}

template <int DT, bool kAligned, int V, int NT>
__global__ void __launch_bounds__(NT) rmsnorm_bwd_kernel(const __grid_constant__ NormBwdArgs a) {
  constexpr int kB = In<DT>::kBytes;
  // As far as the registers last: the next row's loads go out early, dres is
  // read with the others (2048 x 12288 float32: with dres 322 us, late 123).
  constexpr bool kAhead = V * kB <= 4, kLate = V * kB > 8;
  __shared__ float red[2 * kRedWords];
  extern __shared__ __align__(16) float sum_s[];  // [cols], where several groups' dgamma sums meet
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int warp = threadIdx.x >> 5;
  const int group = warp / a.warps;
  const int t = threadIdx.x - group * a.warps * 32;
  const int stride = 256 * a.warps;
  GroupReduce gr{red, a.warps, group, warp - group * a.warps, 0};
  float dg[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[v][i] = 0.0f;
  const float inv_cols = __frcp_rn(float(a.cols));
  const int64_t step = int64_t(gridDim.x) * a.groups;
  Vec8<DT> ny[V], nh[V], nr[V];  // the next row of dy, h and dres
  float nrstd = 0.0f;
  auto load = [&](int64_t row) {
    const int64_t off = row * a.cols * kB;
    nrstd = a.rstd[row];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      ny[v] = load8<DT, kAligned>(a.dy + off, 8 * t + v * stride, a.cols);
      nh[v] = load8<DT, kAligned>(a.h + off, 8 * t + v * stride, a.cols);
      if (!kLate && a.dres != nullptr) nr[v] = load8<DT, kAligned>(a.dres + off, 8 * t + v * stride, a.cols);
    }
  };
  int64_t row = int64_t(blockIdx.x) * a.groups + group;
  if (row < a.rows) load(row);
  for (; row < a.rows; row += step) {
    const int64_t off = row * a.cols * kB;
    const float rstd = nrstd;
    Vec8<DT> dr[V];
    float g[V][8], n[V][8];  // dy * gamma, h * rstd
    float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float gm[8];
      load_gamma8<DT, kAligned>(a.gamma, a.gamma_f32, 8 * t + v * stride, a.cols, gm);
      unpack8<DT>(ny[v], g[v]);
      unpack8<DT>(nh[v], n[v]);
      if (!kLate) dr[v] = nr[v];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        scale2(n[v][i], n[v][i + 1], rstd);
        float x = g[v][i], y = g[v][i + 1];
        mul2(x, y, n[v][i], n[v][i + 1]);
        add2(dg[v][i], dg[v][i + 1], x, y);
        fma2v(x, y, gm[i], gm[i + 1], d0, d1);
        d0 = x, d1 = y;
        mul2(g[v][i], g[v][i + 1], gm[i], gm[i + 1]);
      }
    }
    if (kAhead && row + step < a.rows) load(row + step);
    const float c1 = -(gr.sum(d0 + d1) * inv_cols);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float e[8];
      if (a.dres != nullptr) {
        if (kLate) dr[v] = load8<DT, kAligned>(a.dres + off, 8 * t + v * stride, a.cols);
        unpack8<DT>(dr[v], e);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        fma2(n[v][i], n[v][i + 1], c1, g[v][i], g[v][i + 1]);
        fma2(n[v][i], n[v][i + 1], rstd, e[i], e[i + 1]);
      }
      store8<DT, kAligned>(a.dx + off, 8 * t + v * stride, a.cols, pack8<DT>(n[v]));
    }
    if (!kAhead && row + step < a.rows) load(row + step);
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + int64_t(blockIdx.x) * a.cols;
  if (a.groups > 1) {  // in order; sum_s is a whole number of vectors
    for (int q = 0; q < a.groups; ++q) {
      if (group == q) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = 8 * t + v * stride;
          if (c >= a.cols) continue;
          float4* s = reinterpret_cast<float4*>(sum_s + c);
          if (q > 0) {
            const float4 x = s[0], y = s[1];
            dg[v][0] += x.x, dg[v][1] += x.y, dg[v][2] += x.z, dg[v][3] += x.w;
            dg[v][4] += y.x, dg[v][5] += y.y, dg[v][6] += y.z, dg[v][7] += y.w;
          }
          s[0] = make_float4(dg[v][0], dg[v][1], dg[v][2], dg[v][3]);
          s[1] = make_float4(dg[v][4], dg[v][5], dg[v][6], dg[v][7]);
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) out[c] = sum_s[c];
    return;
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

// How a row is split: `warps` warps of threads with v vectors each, and how
// many rows a block has in work.
struct RowSplit {
  int warps, groups, v;
  int threads() const { return 32 * warps * groups; }
};

RowSplit split_at(int64_t cols, int v, int block_warps) {
  RowSplit s;
  s.v = v;
  s.warps = int(((cols + 7) / 8 + 32 * v - 1) / (32 * v));
  s.groups = std::max(1, block_warps / s.warps);
  return s;
}

// Forward: two vectors per thread (one for a row that fits one warp, four
// above 4096 columns of 16 bits, 8192 of 32), blocks of about eight warps.  8192 x 1536 bf16 with a
// residual, by vectors per thread: one 25.8 us (six warps meet at each row's
// barrier), two 16.9, three 21.2, four 23.7; without the next row's loads
// ahead, two take 20.2.  4096 x 8192: two (sixteen warps) 52.6 us, four 45.9.
RowSplit split_fwd(int64_t cols, int bytes) {
  return split_at(cols, cols <= 256 ? 1 : cols <= (bytes == 4 ? 8192 : 4096) ? 2 : 4, 8);
}

// Backward: one vector per thread while a row's warps fit a block, for the
// dgamma sums and the second pass need the registers, and one large block per
// SM, so that there are few rows of partial sums: 768 threads of 16-bit values
// take 8192 x 1536 in 23.2 us, 512 threads in 37.6 (and 8192 x 1537, whose loads
// spill 12 bytes at 768, in 62.6 and 84.8).  Not by the alignment: which rows a
// thread adds, and so every bit of dgamma, depends on the sizes and the type.
constexpr int bwd_threads(int bytes, int v) { return bytes == 2 && v == 1 ? 768 : 512; }

RowSplit split_bwd(int64_t cols, int bytes) {
  const int v = cols <= 2048 ? 1 : cols <= 8192 ? 2 : 4;
  return split_at(cols, v, bwd_threads(bytes, v) / 32);
}

int norm_shape_check(int dtype, int64_t rows, int64_t cols) {
  if (dtype < FP8_IN_BF16 || dtype > FP8_IN_FP32) return FP8_ERR_INVALID_ARG;
  if (rows < 0 || cols < 1) return FP8_ERR_INVALID_ARG;
  if (cols > kMaxCols || rows > INT32_MAX) return FP8_ERR_UNSUPPORTED;
  return FP8_OK;
}

template <int DT, bool kAligned, int V, int NT>
int launch_fwd1(const NormArgs& a, const RowSplit& s, cudaStream_t st) {
  static int cached[64][kMaxWarps + 1] = {{0}};  // resident blocks per SM by warps per row
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FP8_ERR_CUDA;
  int& bps = cached[dev][s.warps];
  if (bps == 0) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, rmsnorm_kernel<DT, kAligned, V, NT>, s.threads(), 0) !=
            cudaSuccess || n < 1)
      return FP8_ERR_CUDA;
    bps = n;
  }
  const int sms = sm_count_current();
  if (sms < 1) return FP8_ERR_CUDA;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((a.rows + s.groups - 1) / s.groups, int64_t(sms) * bps));
  return launch_pdl(rmsnorm_kernel<DT, kAligned, V, NT>, dim3(unsigned(grid)), dim3(s.threads()), 0, st, 1, a) ==
                 cudaSuccess
             ? FP8_OK
             : FP8_ERR_CUDA;
}

template <int DT, bool kAligned>
int launch_fwd(const NormArgs& a, const RowSplit& s, cudaStream_t st) {
  if (s.v == 4) return launch_fwd1<DT, kAligned, 4, 512>(a, s, st);
  if (s.v == 2)
    return s.threads() > 256 ? launch_fwd1<DT, kAligned, 2, 512>(a, s, st) : launch_fwd1<DT, kAligned, 2, 256>(a, s, st);
  return launch_fwd1<DT, kAligned, 1, 256>(a, s, st);
}

template <int DT, bool kAligned, int V>
int launch_bwd1(const NormBwdArgs& a, const RowSplit& s, int64_t grid, cudaStream_t st) {
  // Shared sums of several groups: at most 8192 columns, since more leave one group.
  const size_t smem = s.groups > 1 ? size_t((a.cols + 7) & ~7) * 4 : 0;
  const cudaError_t e = launch_pdl(rmsnorm_bwd_kernel<DT, kAligned, V, bwd_threads(In<DT>::kBytes, V)>,
                                   dim3(unsigned(grid)), dim3(s.threads()), smem, st, 1, a);
  return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

template <int DT, bool kAligned>
int launch_bwd(const NormBwdArgs& a, const RowSplit& s, int64_t grid, cudaStream_t st) {
  if (s.v == 4) return launch_bwd1<DT, kAligned, 4>(a, s, grid, st);
  if (s.v == 2) return launch_bwd1<DT, kAligned, 2>(a, s, grid, st);
  return launch_bwd1<DT, kAligned, 1>(a, s, grid, st);
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
  const RingWords words(ring_mode ? p->ring : fp8_ring{}, p->amax_out);
  if (!words.aligned()) return FP8_ERR_UNSUPPORTED;
  const size_t n = size_t(p->rows) * size_t(p->cols);
  const Span spans[] = {{p->x, n * eb, false, false, true},
                        {p->residual, n * eb, false, false, true},
                        {p->gamma, size_t(p->cols) * (p->gamma_f32 ? 4 : eb), false, false, false},
                        {p->h, n * eb, true, true, false},
                        {p->y, n * eb, true, true, false},
                        {p->rstd, size_t(p->rows) * 4, true, false, false},
                        {p->codes, n, true, false, false},
                        {p->row_sinv, size_t(p->rows) * 4, true, false, false}};
  if (spans_clash(spans, 8) || words.clash(spans, 8)) return FP8_ERR_INVALID_ARG;
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
  const RowSplit s = split_fwd(p->cols, eb);
  a.warps = s.warps;
  a.groups = s.groups;
  const bool al = p->cols % 8 == 0 && on(p->x, 16) && on(p->residual, 16) && on(p->h, 16) && on(p->y, 16) &&
                  on(p->codes, 8) && on(p->gamma, 16);
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
  const int64_t n = std::min<int64_t>(rows, sms);  // blocks, at most
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
  const bool al = p->cols % 8 == 0 && on(p->dy, 16) && on(p->h, 16) && on(p->dres, 16) && on(p->dx, 16) &&
                  on(p->gamma, 16);
  RowSplit s = split_bwd(p->cols, eb);
  s.groups = int(std::max<int64_t>(1, std::min<int64_t>(s.groups, (p->rows + sms - 1) / sms)));  // few rows: all SMs
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((p->rows + s.groups - 1) / s.groups, sms));
  NormBwdArgs a{};
  a.dy = static_cast<const uint8_t*>(p->dy);
  a.h = static_cast<const uint8_t*>(p->h);
  a.dres = static_cast<const uint8_t*>(p->dres);
  a.rstd = p->rstd;
  a.gamma = p->gamma;
  a.gamma_f32 = p->gamma_f32 != 0 || p->dtype == FP8_IN_FP32;
  a.rows = p->rows;
  a.cols = int(p->cols);
  a.warps = s.warps;
  a.groups = s.groups;
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
  int r;
  switch (p->dtype) {
    case FP8_IN_BF16: r = al ? launch_bwd<FP8_IN_BF16, true>(a, s, grid, st) : launch_bwd<FP8_IN_BF16, false>(a, s, grid, st); break;
    case FP8_IN_FP16: r = al ? launch_bwd<FP8_IN_FP16, true>(a, s, grid, st) : launch_bwd<FP8_IN_FP16, false>(a, s, grid, st); break;
    default: r = al ? launch_bwd<FP8_IN_FP32, true>(a, s, grid, st) : launch_bwd<FP8_IN_FP32, false>(a, s, grid, st); break;
  }
  if (r != FP8_OK || p->dgamma == nullptr || grid == 1) return r;
  return launch_colsum(a.partial, int(grid), p->cols, p->dgamma, st);
}
