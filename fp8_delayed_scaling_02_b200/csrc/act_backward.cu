// fp8_act_backward: the gradient of the product's activation epilogue, cast to
// FP8 for the backward products, with the bias gradients (sm_100a).
//
// A stream bound by HBM: with a gate, three reads of 2 bytes and two code
// bytes per element; the activation's two fast-math operations hide behind it.
// One pass computes both gradients, their casts, their amaxes (each folded
// into its own ring by the last block) and, where wanted, the column sums.
//   * Without sums the tensors are one flat run of 8-element vectors, two in
//     flight per thread, over one wave of resident blocks.
//   * With sums a block owns a strip of 256 columns (or 64) and walks down its
//     rows, so a thread's 8 columns stay fixed and their sums in registers;
//     strips are cut into row chunks to fill one wave, each chunk writes one
//     float32 row of partial sums, and a second launch adds those in order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "activation.cuh"
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

constexpr int kAbThreads = 256;
constexpr int kMaxStripCols = 256;
// Blocks per SM of the kernels with sums, and so the registers they may use.  At
// this count some spill (16 bits with a gate 24 bytes a thread, unaligned 48;
// float32 16 to 56); one block fewer does not.  us here / one block fewer: gated bf16 8192 x 4096 54.3 /
// 60.2, 8192 x 1537 58.9 / 71.9, 512 x 4096 10.5 / 9.5; without a gate bf16 8192 x
// 4096 40.6 / 47.3, 512 x 4096 6.9 / 7.2, float32 8192 x 4096 42.8 / 43.5, 1000 x 1537
// 9.2 / 7.9.
constexpr int sum_blocks(bool gate) { return gate ? 3 : 4; }

struct ActBwdArgs {
  const uint8_t* dy;
  const uint8_t* z;
  const uint8_t* u;
  int64_t rows, cols, n;
  int act, fmt;
  RingArgs ring, ring_u;
  uint8_t* dzq;
  uint8_t* duq;
  int64_t strips;    // with sums: blockIdx.x = chunk * strips + strip
  int log_lanes;     // threads across a strip, 8 columns each: 8 or 32
  int64_t chunks;
  float* part;       // [chunks][cols] sums of dz
  float* part_u;     // and of du
};

template <int DT, bool kGate>
struct Grads {
  Vec8<DT> dy;
  Vec8<FP8_IN_BF16> z, u;
};

// Vector `c` of the row at element `e` (both in elements), `cols` long.
template <int DT, bool kAligned, bool kGate>
__device__ __forceinline__ void load_grads(const ActBwdArgs& a, int64_t e, int c, int cols, Grads<DT, kGate>& g) {
  g.dy = load8<DT, kAligned>(a.dy + e * In<DT>::kBytes, c, cols);
  if (a.z != nullptr) g.z = load8<FP8_IN_BF16, kAligned>(a.z + 2 * e, c, cols);
  if constexpr (kGate) g.u = load8<FP8_IN_BF16, kAligned>(a.u + 2 * e, c, cols);
}

__device__ __forceinline__ void codes8(const float (&v)[8], int fmt, float s, uint32_t& lo, uint32_t& hi) {
  if (fmt == FP8_E5M2) {
    lo = cvt4<FP8_E5M2>(v[0], v[1], v[2], v[3], s);
    hi = cvt4<FP8_E5M2>(v[4], v[5], v[6], v[7], s);
  } else {
    lo = cvt4<FP8_E4M3>(v[0], v[1], v[2], v[3], s);
    hi = cvt4<FP8_E4M3>(v[4], v[5], v[6], v[7], s);
  }
}

template <int ACT>
__device__ __forceinline__ void slopes8(float (&z)[8], float (&sl)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) act_slope_pair<ACT>(z[i], z[i + 1], sl[i], sl[i + 1]);
}

// dz (and du) of one vector: codes out, |.| into the amaxes, values into the
// sums.  Lanes beyond the row's end hold dy = 0, hence dz = du = 0.
template <int DT, bool kAligned, bool kGate, bool kDb>
__device__ __forceinline__ void emit_grads(const ActBwdArgs& a, int64_t e, int c, int cols, const Grads<DT, kGate>& g,
                                           float s, float su, float& amax, float& amax_u, float (&sum)[8],
                                           float (&sum_u)[8]) {
  float d[8], z[8], u[8], w[8], sl[8];
  unpack8<DT>(g.dy, d);
  if (a.z != nullptr) {
    unpack8<FP8_IN_BF16>(g.z, z);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = 0.0f;
  }
  switch (a.act) {  // uniform; z becomes act(z)
    case FP8_ACT_RELU: slopes8<FP8_ACT_RELU>(z, sl); break;
    case FP8_ACT_GELU: slopes8<FP8_ACT_GELU>(z, sl); break;
    case FP8_ACT_SILU: slopes8<FP8_ACT_SILU>(z, sl); break;
    default: slopes8<FP8_ACT_NONE>(z, sl);
  }
  if constexpr (kGate) {
    unpack8<FP8_IN_BF16>(g.u, u);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      w[i] = d[i], w[i + 1] = d[i + 1];
      mul2(w[i], w[i + 1], z[i], z[i + 1]);
      mul2(d[i], d[i + 1], u[i], u[i + 1]);
    }
  }
  if (a.act == FP8_ACT_RELU) {  // nothing passes where the slope is 0, not even 0 times an infinity
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = sl[i] == 0.0f ? 0.0f : d[i];
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    mul2(d[i], d[i + 1], sl[i], sl[i + 1]);
    amax = fmaxf(amax, fmaxf(fabsf(d[i]), fabsf(d[i + 1])));
    if constexpr (kGate) amax_u = fmaxf(amax_u, fmaxf(fabsf(w[i]), fabsf(w[i + 1])));
    if constexpr (kDb) add2(sum[i], sum[i + 1], d[i], d[i + 1]);
    if constexpr (kDb && kGate) add2(sum_u[i], sum_u[i + 1], w[i], w[i + 1]);
  }
  uint32_t lo, hi;
  codes8(d, a.fmt, s, lo, hi);
  store8_codes<kAligned>(a.dzq + e, c, cols, lo, hi);
  if constexpr (kGate) {
    codes8(w, a.fmt, su, lo, hi);
    store8_codes<kAligned>(a.duq + e, c, cols, lo, hi);
  }
}

// One thread's share of a block's end of work on a ring (threads 0..16 hold
// the first ring's history and idx, threads 32..48 the second's).
__device__ __forceinline__ void commit_ring(const ActBwdArgs& a, const RingArgs& r, float m, float s, float* hist,
                                            int idx) {
  if (a.fmt == FP8_E5M2) commit_block_amax<FP8_E5M2>(m, r, s, hist, idx, gridDim.x);
  else commit_block_amax<FP8_E4M3>(m, r, s, hist, idx, gridDim.x);
}

template <int DT, bool kAligned, bool kGate, bool kDb>
__global__ void __launch_bounds__(kAbThreads, kDb ? sum_blocks(kGate) : 3) act_backward_kernel(const __grid_constant__ ActBwdArgs a) {
  __shared__ float warp_max[2][kAbThreads / 32];
  __shared__ float hist_s[2][kHistoryLen];
  __shared__ int idx_s[2];
  __shared__ float sum_s[kDb ? (kGate ? 2 : 1) * (kAbThreads / 32) * kMaxStripCols : 1];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float s = *a.ring.scale;
  const float su = kGate ? *a.ring_u.scale : 1.0f;
  if (warp < (kGate ? 2 : 1)) {  // neither ring is written before the last block's fold
    const RingArgs& r = warp == 0 ? a.ring : a.ring_u;
    if (r.amax_out == nullptr) {
      if (lane < kHistoryLen) hist_s[warp][lane] = r.history[lane];
      if (lane == kHistoryLen) idx_s[warp] = *r.idx;
    }
  }
  float amax = 0.0f, amax_u = 0.0f;
  float sum[8], sum_u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = sum_u[i] = 0.0f;
  Grads<DT, kGate> g0, g1;

  if constexpr (kDb) {
    const int64_t chunk = blockIdx.x / a.strips, strip = blockIdx.x - chunk * a.strips;
    const int cols = int(a.cols);
    const int lanes = 1 << a.log_lanes;
    const int c = int(strip) * 8 * lanes + 8 * (threadIdx.x & (lanes - 1));
    const int rows = kAbThreads >> a.log_lanes;  // of one step of a block
    const int64_t step = a.chunks * rows;
    for (int64_t r = chunk * rows + (threadIdx.x >> a.log_lanes); r < a.rows; r += 2 * step) {
      const bool two = r + step < a.rows;
      load_grads<DT, kAligned>(a, r * a.cols, c, cols, g0);
      if (two) load_grads<DT, kAligned>(a, (r + step) * a.cols, c, cols, g1);
      emit_grads<DT, kAligned, kGate, kDb>(a, r * a.cols, c, cols, g0, s, su, amax, amax_u, sum, sum_u);
      if (two) emit_grads<DT, kAligned, kGate, kDb>(a, (r + step) * a.cols, c, cols, g1, s, su, amax, amax_u, sum, sum_u);
    }
    // A warp's rows by shuffles (narrow strips), the warps through shared memory, in order.
    if (lanes == 8) {
#pragma unroll
      for (int o = 8; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], o);
          if constexpr (kGate) sum_u[i] += __shfl_xor_sync(0xFFFFFFFFu, sum_u[i], o);
        }
    }
    if (lane < lanes) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum_s[warp * kMaxStripCols + 8 * lane + i] = sum[i];
        if constexpr (kGate) sum_s[(kAbThreads / 32 + warp) * kMaxStripCols + 8 * lane + i] = sum_u[i];
      }
    }
  } else {
    const int64_t nvec = (a.n + 7) / 8;
    const int64_t nthr = int64_t(gridDim.x) * kAbThreads;
    for (int64_t j = int64_t(blockIdx.x) * kAbThreads + threadIdx.x; j < nvec; j += 2 * nthr) {
      const int64_t j1 = j + nthr;
      const int m0 = int(min(int64_t(8), a.n - 8 * j)), m1 = int(min(int64_t(8), a.n - 8 * j1));
      load_grads<DT, kAligned>(a, 8 * j, 0, m0, g0);
      if (j1 < nvec) load_grads<DT, kAligned>(a, 8 * j1, 0, m1, g1);
      emit_grads<DT, kAligned, kGate, kDb>(a, 8 * j, 0, m0, g0, s, su, amax, amax_u, sum, sum_u);
      if (j1 < nvec) emit_grads<DT, kAligned, kGate, kDb>(a, 8 * j1, 0, m1, g1, s, su, amax, amax_u, sum, sum_u);
    }
  }

#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if constexpr (kGate) amax_u = fmaxf(amax_u, __shfl_xor_sync(0xFFFFFFFFu, amax_u, o));
  }
  if (lane == 0) {
    warp_max[0][warp] = amax;
    warp_max[1][warp] = amax_u;
  }
  __syncthreads();
  if (lane == 0 && warp < (kGate ? 2 : 1)) {
    float m = 0.0f;
#pragma unroll
    for (int w = 0; w < kAbThreads / 32; ++w) m = fmaxf(m, warp_max[warp][w]);
    commit_ring(a, warp == 0 ? a.ring : a.ring_u, m, warp == 0 ? s : su, hist_s[warp], idx_s[warp]);
  }
  if constexpr (kDb) {
    const int64_t chunk = blockIdx.x / a.strips, strip = blockIdx.x - chunk * a.strips;
    const int width = 8 << a.log_lanes;
    const int64_t c = strip * width + threadIdx.x;
    if (threadIdx.x < width && c < a.cols) {
#pragma unroll
      for (int k = 0; k < (kGate ? 2 : 1); ++k) {
        float* out = k == 0 ? a.part : a.part_u;
        if (out == nullptr) continue;
        float r = 0.0f;
#pragma unroll
        for (int w = 0; w < kAbThreads / 32; ++w) r += sum_s[(k * (kAbThreads / 32) + w) * kMaxStripCols + threadIdx.x];
        out[chunk * a.cols + c] = r;
      }
    }
  }
}

// ---- host side -----------------------------------------------------------------

// Threads across a strip and row chunks per strip.
//   * Up to kFewRows rows: narrow strips of one chunk, whose sums are the
//     result (128 x 4096 gated: 6.9 us, in two launches 8.7).
//   * More: as many chunks as fit in one wave together, of at least two steps
//     each.  With a gate strips are as wide as a warp, unless that wastes over a
//     sixteenth of the strips' columns (1537 columns: 7 strips of 256 for 6, 25
//     of 64 for 24): 8192 x 4096 takes 53.6 us, in strips of 64 columns 65.9.
//     Without, the fewer rows of partial sums of narrow strips count for more:
//     512 x 4096 6.7 us, in strips of 256 7.6; 8192 x 1536 18.4 and 19.1.
constexpr int64_t kFewRows = 256;

int lanes_of(int64_t rows, int64_t cols, bool gate) {
  const int64_t wide = (cols + 255) / 256 * 256;
  return gate && rows > kFewRows && wide - cols <= cols / 16 ? 32 : 8;
}

int64_t strips_of(int64_t cols, int lanes) { return (cols + 8 * lanes - 1) / (8 * lanes); }

int64_t chunks_of(int64_t rows, int64_t cols, bool gate, int sms) {
  if (rows <= kFewRows) return 1;
  const int lanes = lanes_of(rows, cols, gate);
  const int64_t fit = int64_t(sms) * sum_blocks(gate) / std::max<int64_t>(1, strips_of(cols, lanes));
  return std::max<int64_t>(1, std::min<int64_t>(fit, rows / (2 * kAbThreads / lanes)));
}

template <int DT, bool kAligned, bool kGate, bool kDb>
int launch_ab1(ActBwdArgs a, int sms, cudaStream_t st) {
  int64_t grid;
  if (kDb) {
    grid = a.strips * a.chunks;
  } else {
    static int cached[64] = {0};
    const int bps = resident_blocks(act_backward_kernel<DT, kAligned, kGate, kDb>, kAbThreads, cached);
    if (bps < 1) return FP8_ERR_CUDA;
    const int64_t vecs = (a.n + 7) / 8;
    grid = std::max<int64_t>(1, std::min<int64_t>((vecs + kAbThreads - 1) / kAbThreads, int64_t(sms) * bps));
  }
  return launch_pdl(act_backward_kernel<DT, kAligned, kGate, kDb>, dim3(unsigned(grid)), dim3(kAbThreads), 0, st, 1,
                    a) == cudaSuccess
             ? FP8_OK
             : FP8_ERR_CUDA;
}

template <int DT, bool kAligned>
int launch_ab(const ActBwdArgs& a, bool gate, bool db, int sms, cudaStream_t st) {
  if (gate) return db ? launch_ab1<DT, kAligned, true, true>(a, sms, st) : launch_ab1<DT, kAligned, true, false>(a, sms, st);
  return db ? launch_ab1<DT, kAligned, false, true>(a, sms, st) : launch_ab1<DT, kAligned, false, false>(a, sms, st);
}

int ring_check(const fp8_ring& r, const float* amax_out) {
  if (!r.scale || !r.scale_inv || !r.scratch || (amax_out == nullptr && (!r.history || !r.idx)))
    return FP8_ERR_INVALID_ARG;
  return on(r.scratch, 8) ? FP8_OK : FP8_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace fp8ds

using namespace fp8ds;

extern "C" size_t fp8_act_backward_workspace_bytes(int64_t rows, int64_t cols, int gated) {
  if (rows <= 0 || cols <= 0 || cols > (int64_t(1) << 30) || rows > INT32_MAX) return 0;
  const int sms = sm_count_current();
  if (sms <= 0) return 0;
  const int64_t chunks = chunks_of(rows, cols, gated != 0, sms);
  return chunks > 1 ? size_t(chunks) * size_t(cols) * 4 * (gated ? 2 : 1) : 0;
}

extern "C" int fp8_act_backward(const fp8_act_backward_args* p, fp8_stream_t stream) {
  if (p == nullptr) return FP8_ERR_INVALID_ARG;
  if (p->dtype < FP8_IN_BF16 || p->dtype > FP8_IN_FP32 || p->rows < 0 || p->cols < 0) return FP8_ERR_INVALID_ARG;
  if (p->act < FP8_ACT_NONE || p->act > FP8_ACT_SILU || (p->fmt != FP8_E4M3 && p->fmt != FP8_E5M2))
    return FP8_ERR_INVALID_ARG;
  const bool gate = p->u != nullptr || p->duq != nullptr;
  const bool some = p->rows > 0 && p->cols > 0;
  if (some && (p->dy == nullptr || p->dzq == nullptr)) return FP8_ERR_INVALID_ARG;
  if (some && gate && (p->u == nullptr || p->duq == nullptr)) return FP8_ERR_INVALID_ARG;
  if (some && p->z == nullptr && (gate || p->act != FP8_ACT_NONE)) return FP8_ERR_INVALID_ARG;
  const bool ring_u = p->ring_u.scale != nullptr;
  if (some && gate != ring_u) return FP8_ERR_INVALID_ARG;
  if (p->amax_out_u != nullptr && (!ring_u || p->amax_out_u == p->amax_out)) return FP8_ERR_INVALID_ARG;
  if (p->dbu != nullptr && (p->db == nullptr || !ring_u)) return FP8_ERR_INVALID_ARG;
  int rc = ring_check(p->ring, p->amax_out);
  if (rc == FP8_OK && ring_u) rc = ring_check(p->ring_u, p->amax_out_u);
  if (rc == FP8_ERR_INVALID_ARG) return rc;
  const RingWords words(p->ring, p->amax_out), words_u(ring_u ? p->ring_u : fp8_ring{}, p->amax_out_u);
  if (words.clash(words_u)) return FP8_ERR_INVALID_ARG;
  if (rc != FP8_OK) return rc;
  if (p->cols > (int64_t(1) << 30) || p->rows > INT32_MAX) return FP8_ERR_UNSUPPORTED;
  const int eb = p->dtype == FP8_IN_FP32 ? 4 : 2;
  if (!on(p->dy, eb) || !on(p->z, 2) || !on(p->u, 2) || !on(p->db, 4) || !on(p->dbu, 4) || !on(p->workspace, 4) ||
      !words.aligned() || !words_u.aligned())
    return FP8_ERR_UNSUPPORTED;
  const size_t n = size_t(p->rows) * size_t(p->cols);
  const Span spans[] = {{p->dy, n * eb, false, false, false},
                        {p->z, n * 2, false, false, false},
                        {p->u, n * 2, false, false, false},
                        {p->dzq, n, true, false, false},
                        {p->duq, n, true, false, false},
                        {p->db, size_t(p->cols) * 4, true, false, false},
                        {p->dbu, size_t(p->cols) * 4, true, false, false},
                        {p->workspace, p->db ? p->workspace_bytes : 0, true, false, false}};
  if (spans_clash(spans, 8) || words.clash(spans, 8) || words_u.clash(spans, 8)) return FP8_ERR_INVALID_ARG;
  const int sms = sm_count_current();
  if (sms <= 0) return FP8_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ActBwdArgs a{};
  a.dy = static_cast<const uint8_t*>(p->dy);
  a.z = static_cast<const uint8_t*>(p->z);
  a.u = static_cast<const uint8_t*>(p->u);
  a.rows = p->rows;
  a.cols = p->cols;
  a.n = p->rows * p->cols;
  a.act = p->act;
  a.fmt = p->fmt;
  a.ring = RingArgs{p->ring.history, p->ring.idx, p->ring.scale, p->ring.scale_inv, p->ring.scratch, p->amax_out};
  if (ring_u)
    a.ring_u = RingArgs{p->ring_u.history, p->ring_u.idx, p->ring_u.scale, p->ring_u.scale_inv, p->ring_u.scratch,
                        p->amax_out_u};
  a.dzq = p->dzq;
  a.duq = p->duq;
  const bool db = p->db != nullptr && some;
  if (db) {
    const int lanes = lanes_of(p->rows, p->cols, ring_u);
    a.log_lanes = lanes == 32 ? 5 : 3;
    a.strips = strips_of(p->cols, lanes);
    a.chunks = chunks_of(p->rows, p->cols, ring_u, sms);
    a.part = p->db;  // one chunk: its sums are the result
    a.part_u = p->dbu;
    if (a.chunks > 1) {
      const size_t each = size_t(a.chunks) * size_t(p->cols) * 4;
      if (p->workspace == nullptr || p->workspace_bytes < each * (p->dbu ? 2 : 1)) return FP8_ERR_INVALID_ARG;
      a.part = static_cast<float*>(p->workspace);
      a.part_u = p->dbu ? a.part + size_t(a.chunks) * size_t(p->cols) : nullptr;
    }
  }
  // Vectors never straddle a 16-byte boundary when the bases are aligned and a
  // row (with sums) or the whole run (without) is a whole number of them.
  const bool al = (db ? p->cols : a.n) % 8 == 0 && on(p->dy, 16) && on(p->z, 16) && on(p->u, 16) && on(p->dzq, 8) &&
                  on(p->duq, 8);
  switch (p->dtype) {
    case FP8_IN_BF16: rc = al ? launch_ab<FP8_IN_BF16, true>(a, ring_u, db, sms, st) : launch_ab<FP8_IN_BF16, false>(a, ring_u, db, sms, st); break;
    case FP8_IN_FP16: rc = al ? launch_ab<FP8_IN_FP16, true>(a, ring_u, db, sms, st) : launch_ab<FP8_IN_FP16, false>(a, ring_u, db, sms, st); break;
    default: rc = al ? launch_ab<FP8_IN_FP32, true>(a, ring_u, db, sms, st) : launch_ab<FP8_IN_FP32, false>(a, ring_u, db, sms, st); break;
  }
  if (rc != FP8_OK || p->db == nullptr) return rc;
  const int parts = db ? int(a.chunks) : 0;
  if (parts != 1) {
    rc = launch_colsum(a.part, parts, p->cols, p->db, st);
    if (rc == FP8_OK && p->dbu != nullptr) rc = launch_colsum(a.part_u, parts, p->cols, p->dbu, st);
  }
  return rc;
}
