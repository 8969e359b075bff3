// fp8_mm_act for a few rows of A: the products of single decoded tokens.
//
// Reading the weight B once is all there is to do (6.3 MB and 13 MFLOP for one
// token at N = 4096, K = 1536), so B goes from global memory straight into the
// registers of the MMA that uses it: no tile, no shared memory, and as many
// 16-byte loads in flight as the SM has warps for.
//   * A block owns 16 rows of B; its warps take turns along K, 64 bytes of each
//     row a step.  B is the row operand of mma m16n8k32 and the tokens, eight
//     at a time, its column operand (M of 128 would leave 15/16 of a tcgen05
//     tile's rows empty, and the tile kernel reads 64 rows of B per SM in
//     sequence: 8.0 us at the sizes above).
//   * A lane's 16 bytes at k0 + 16 (lane % 4) serve as four of the fragments'
//     32-bit words.  Which k a word stands for is the same on both sides, and
//     the order of a sum's terms is free.
//   * The warps' partial sums meet in shared memory, in order; then scale,
//     bias, activation, operand and the cast, 16 contiguous outputs per token.
// FP8 operands are exact in the products and the sums are float32.
#include <cuda_bf16.h>

#include <algorithm>

#include "activation.cuh"
#include "amax_fold.cuh"
#include "common.cuh"
#include "fp8_ring.cuh"
#include "mm_act.cuh"

namespace fp8ds {
namespace {

constexpr int kSkThreads = 256;
constexpr int kSkWarps = kSkThreads / 32;
constexpr int kSkRows = 16;   // rows of B per block
constexpr int kSkUnroll = 4;  // steps of 64 bytes in flight per warp

template <int FA, int FB>
__device__ __forceinline__ void mma_f8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
#define FP8DS_MMA(ta, tb)                                                              \
  asm volatile("mma.sync.aligned.m16n8k32.row.col.f32." ta "." tb ".f32 "              \
               "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"                 \
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                        \
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if constexpr (FA == FP8_E4M3 && FB == FP8_E4M3) FP8DS_MMA("e4m3", "e4m3");
  else if constexpr (FA == FP8_E4M3) FP8DS_MMA("e4m3", "e5m2");
  else if constexpr (FB == FP8_E4M3) FP8DS_MMA("e5m2", "e4m3");
  else FP8DS_MMA("e5m2", "e5m2");
#undef FP8DS_MMA
}

// NT: groups of eight tokens.  FB is the format of B, the MMA's row operand.
template <int FA, int FB, int NT, bool kOut8>
__global__ void __launch_bounds__(kSkThreads) mm_skinny_kernel(const __grid_constant__ SkinnyArgs p) {
  constexpr int kPitch = 8 * NT + 4;  // floats between rows of the partial sums: conflict-free for the fragments
  __shared__ float red[kSkWarps][kSkRows][kPitch];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = int(blockIdx.x) * kSkRows;
  const float s_out = kOut8 ? *p.ring.scale : 0.0f;
  RingCache rc{0.0f, 0};
  if constexpr (kOut8) rc = prefetch_ring(p.ring);

  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
  const uint8_t* b0p = p.B + int64_t(n0 + g) * p.K + 16 * t;
  const uint8_t* b1p = b0p + int64_t(8) * p.K;
  const uint8_t* ap = p.A + int64_t(g) * p.K + 16 * t;
  const bool b0_ok = n0 + g < p.N, b1_ok = n0 + g + 8 < p.N;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int steps = (p.K + 63) / 64;
  for (int s0 = warp; s0 < steps; s0 += kSkWarps * kSkUnroll) {
    uint4 wb0[kSkUnroll], wb1[kSkUnroll], wa[kSkUnroll][NT];
#pragma unroll
    for (int u = 0; u < kSkUnroll; ++u) {
      const int k = 64 * (s0 + u * kSkWarps);
      const bool k_ok = k + 16 * t < p.K;
      wb0[u] = b0_ok && k_ok ? __ldg(reinterpret_cast<const uint4*>(b0p + k)) : zero;
      wb1[u] = b1_ok && k_ok ? __ldg(reinterpret_cast<const uint4*>(b1p + k)) : zero;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        wa[u][j] = k_ok && 8 * j + g < p.M ? __ldg(reinterpret_cast<const uint4*>(ap + int64_t(8 * j) * p.K + k)) : zero;
    }
#pragma unroll
    for (int u = 0; u < kSkUnroll; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mma_f8<FB, FA>(acc[j], wb0[u].x, wb1[u].x, wb0[u].y, wb1[u].y, wa[u][j].x, wa[u][j].y);
        mma_f8<FB, FA>(acc[j], wb0[u].z, wb1[u].z, wb0[u].w, wb1[u].w, wa[u][j].z, wa[u][j].w);
      }
  }
  // acc[j]: rows g and g + 8 of B, tokens 8j + 2t and + 1.
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    red[warp][g][8 * j + 2 * t] = acc[j][0];
    red[warp][g][8 * j + 2 * t + 1] = acc[j][1];
    red[warp][g + 8][8 * j + 2 * t] = acc[j][2];
    red[warp][g + 8][8 * j + 2 * t + 1] = acc[j][3];
  }
  __syncthreads();

  float amax = 0.0f;
  const int n = n0 + (threadIdx.x & 15);
  const float sinv_b = *p.sinv_b;
  const float bias = p.bias != nullptr && n < p.N ? __ldg(p.bias + n) : 0.0f;
  for (int m = threadIdx.x >> 4; m < p.M; m += kSkThreads / 16) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kSkWarps; ++w) v += red[w][threadIdx.x & 15][m];
    if (n < p.N) {
      const int64_t o = int64_t(m) * p.N + n;
      const float sab = __fmul_rn(p.sinv_a[p.a_rows ? m : 0], sinv_b);
      const float z = fmaf(v, sab, bias);
      if (p.z != nullptr) p.z[o] = __bfloat16_as_ushort(__float2bfloat16_rn(z));
      float y = act_value(p.act, z);
      if (p.aux != nullptr) {
        const float x = __uint_as_float(uint32_t(p.aux[o]) << 16);
        y = p.aux_mul ? __fmul_rn(y, x) : __fadd_rn(y, x);
      }
      if constexpr (kOut8) {
        amax = fmaxf(amax, fabsf(y));
        p.out8[o] = p.out_fmt == FP8_E5M2 ? cvt_one<FP8_E5M2>(y, s_out) : cvt_one<FP8_E4M3>(y, s_out);
      } else {
        p.out[o] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
      }
    }
  }
  if constexpr (kOut8) {
    if (p.out_fmt == FP8_E5M2) amax_ticket_fold<FP8_E5M2, kSkThreads>(amax, p.ring, s_out, rc, gridDim.x);
    else amax_ticket_fold<FP8_E4M3, kSkThreads>(amax, p.ring, s_out, rc, gridDim.x);
  }
}

template <int FA, int FB, int NT>
cudaError_t launch_nt(const SkinnyArgs& a, cudaStream_t st) {
  const dim3 grid(unsigned((a.N + kSkRows - 1) / kSkRows));
  if (a.out8 != nullptr) return launch_pdl(mm_skinny_kernel<FA, FB, NT, true>, grid, dim3(kSkThreads), 0, st, 1, a);
  return launch_pdl(mm_skinny_kernel<FA, FB, NT, false>, grid, dim3(kSkThreads), 0, st, 1, a);
}

template <int FA, int FB>
cudaError_t launch_fmt(const SkinnyArgs& a, cudaStream_t st) {
  if (a.M <= 8) return launch_nt<FA, FB, 1>(a, st);
  if (a.M <= 16) return launch_nt<FA, FB, 2>(a, st);
  return launch_nt<FA, FB, 4>(a, st);
}

}  // namespace

int launch_skinny(const SkinnyArgs& a, cudaStream_t st) {
  cudaError_t e;
  if (a.fmt_a == FP8_E4M3)
    e = a.fmt_b == FP8_E4M3 ? launch_fmt<FP8_E4M3, FP8_E4M3>(a, st) : launch_fmt<FP8_E4M3, FP8_E5M2>(a, st);
  else
    e = a.fmt_b == FP8_E4M3 ? launch_fmt<FP8_E5M2, FP8_E4M3>(a, st) : launch_fmt<FP8_E5M2, FP8_E5M2>(a, st);
  return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

}  // namespace fp8ds
