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

// NT: groups of eight tokens.  RG: groups of sixteen rows of B per block.  FB is the format of B, the MMA's row operand.
template <int FA, int FB, int NT, int RG, bool kOut8>
__global__ void __launch_bounds__(kSkThreads) mm_skinny_kernel(const __grid_constant__ SkinnyArgs p) {
  constexpr int kUnroll = RG * NT >= 4 ? 2 : 4;  // steps of 64 bytes in flight per warp
  constexpr int kPitch = 8 * NT + 4;  // floats between rows of the partial sums: conflict-free for the fragments
  __shared__ float red[kSkWarps][16 * RG][kPitch];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = int(blockIdx.x) * 16 * RG;
  const float s_out = kOut8 ? *p.ring.scale : 0.0f;
  RingCache rc{0.0f, 0};
  if constexpr (kOut8) rc = prefetch_ring(p.ring);

  float acc[RG][NT][4];
#pragma unroll
  for (int q = 0; q < RG; ++q)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[q][j][0] = acc[q][j][1] = acc[q][j][2] = acc[q][j][3] = 0.0f;
  const uint8_t* bp = p.B + int64_t(n0 + g) * p.K + 16 * t;
  const uint8_t* ap = p.A + int64_t(g) * p.K + 16 * t;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int steps = (p.K + 63) / 64;
  for (int s0 = warp; s0 < steps; s0 += kSkWarps * kUnroll) {
    uint4 wb[kUnroll][2 * RG], wa[kUnroll][NT];  // rows g, g + 8, g + 16, ...; tokens g, g + 8, ...
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = 64 * (s0 + u * kSkWarps);
      const bool k_ok = k + 16 * t < p.K;
#pragma unroll
      for (int q = 0; q < 2 * RG; ++q)
        wb[u][q] = k_ok && n0 + g + 8 * q < p.N
                       ? __ldg(reinterpret_cast<const uint4*>(bp + int64_t(8 * q) * p.K + k)) : zero;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        wa[u][j] = k_ok && 8 * j + g < p.M ? __ldg(reinterpret_cast<const uint4*>(ap + int64_t(8 * j) * p.K + k)) : zero;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int q = 0; q < RG; ++q) {
        const uint4 lo = wb[u][2 * q], hi = wb[u][2 * q + 1];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma_f8<FB, FA>(acc[q][j], lo.x, hi.x, lo.y, hi.y, wa[u][j].x, wa[u][j].y);
          mma_f8<FB, FA>(acc[q][j], lo.z, hi.z, lo.w, hi.w, wa[u][j].z, wa[u][j].w);
        }
      }
  }
  // acc[q][j]: rows 16q + g and + 8 of B, tokens 8j + 2t and + 1.
#pragma unroll
  for (int q = 0; q < RG; ++q)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      red[warp][16 * q + g][8 * j + 2 * t] = acc[q][j][0];
      red[warp][16 * q + g][8 * j + 2 * t + 1] = acc[q][j][1];
      red[warp][16 * q + g + 8][8 * j + 2 * t] = acc[q][j][2];
      red[warp][16 * q + g + 8][8 * j + 2 * t + 1] = acc[q][j][3];
    }
  __syncthreads();

  float amax = 0.0f;
  const int col = threadIdx.x % (16 * RG), n = n0 + col;
  const float sinv_b = *p.sinv_b;
  const float bias = p.bias != nullptr && n < p.N ? __ldg(p.bias + n) : 0.0f;
  for (int m = threadIdx.x / (16 * RG); m < p.M; m += kSkThreads / (16 * RG)) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kSkWarps; ++w) v += red[w][col][m];
    if (n < p.N) {
      const int64_t o = int64_t(m) * p.N + n;
      const float sab = __fmul_rn(p.sinv_a[p.a_rows ? m : 0], sinv_b);
      const float z = fmaf(v, sab, bias);
      if (p.z != nullptr) p.z[o] = __bfloat16_as_ushort(__float2bfloat16_rn(z));
      float y = act_one(p.act, z);
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

template <int FA, int FB, int NT, int RG>
cudaError_t launch_rg(const SkinnyArgs& a, cudaStream_t st) {
  const dim3 grid(unsigned((a.N + 16 * RG - 1) / (16 * RG)));
  if (a.out8 != nullptr) return launch_pdl(mm_skinny_kernel<FA, FB, NT, RG, true>, grid, dim3(kSkThreads), 0, st, 1, a);
  return launch_pdl(mm_skinny_kernel<FA, FB, NT, RG, false>, grid, dim3(kSkThreads), 0, st, 1, a);
}

// Two groups of rows where that still leaves a block for every SM: the tokens
// are read and converted half as often (one token at 8192 x 4096: 7.9 us, one
// group 8.7; at 4096 x 1536 3.7 and 3.1).
template <int FA, int FB>
cudaError_t launch_fmt(const SkinnyArgs& a, int sms, cudaStream_t st) {
  const bool two = (a.N + 31) / 32 >= sms;
  if (a.M <= 8) return two ? launch_rg<FA, FB, 1, 2>(a, st) : launch_rg<FA, FB, 1, 1>(a, st);
  if (a.M <= 16) return two ? launch_rg<FA, FB, 2, 2>(a, st) : launch_rg<FA, FB, 2, 1>(a, st);
  return launch_rg<FA, FB, 4, 1>(a, st);
}

}  // namespace

// The FP8 mma of mma.sync converts its operands first, at a rate that more
// tokens and longer rows soon reach: a block's time grows with K and with every
// eight tokens.  The tile kernels take the same time up to 32 tokens and, where a
// tile's K can be split, little more for a longer one.  us here / there, by N x K:
//                   8 tokens      16 tokens     32 tokens
//   512 x 512       2.2 /  5.2    2.7 /  5.3    3.6 /  5.3
//   1536 x 1536     3.0 /  5.0    3.9 /  5.1    6.1 /  5.4
//   4096 x 1536     3.5 /  6.3    4.2 /  6.3    6.6 /  6.4
//   1536 x 4096     4.8 /  6.0    6.6 /  6.0   10.3 /  6.0
//   4096 x 4096     5.5 /  7.9    6.9 /  8.2   11.2 /  7.3
//   8192 x 4096     8.6 / 13.7   15.2 / 13.9   33.2 / 12.0
//   1536 x 8192     7.9 /  6.9   11.4 /  6.7   18.1 /  7.1
//   1024 x 16384    9.6 /  8.5   16.9 /  8.7   32.1 /  8.9
// Up to 16 tokens K decides; above 8, sooner with few columns, whose tiles split
// deepest (1536 x 3328: 1.03 of the tiles' time, 2048 x 4096: 1.00), and with many,
// by the size of the weight.  Above 16 tokens the blocks have to be resident at
// once, three to an SM (32 tokens, 7040 x 2048: 7.0 / 8.8, 7168 x 2048: 11.7 / 8.9),
// and K is short, but where 64-column tiles are too many for a pair of CTAs each
// (4224 x 2048: 7.1 / 6.6, 4352 x 2048: 7.2 / 7.8).  Over 880 sizes measured (N of 256
// to 16384, K of 256 to 16384) the kernel taken is at most 6% slower than the
// other at all but eleven, and 16% at the worst of those (1536 x 8192, 8 tokens).
bool skinny_wins(int64_t M, int64_t N, int64_t K, int sms) {
  constexpr int64_t kPairedBlocks = 264;  // of 16 columns: 66 tiles of 64
  const int64_t blocks = (N + 15) / 16;
  if (M <= 8) return K <= 8192;
  if (M <= 16) return K <= (N <= 1536 ? 3328 : 4096) && N * K < (int64_t(22) << 20);
  return M <= kSkinnyMaxM && blocks <= 3 * int64_t(sms) && K <= (blocks > kPairedBlocks ? 2560 : 1024);
}

int launch_skinny(const SkinnyArgs& a, int sms, cudaStream_t st) {
  cudaError_t e;
  if (a.fmt_a == FP8_E4M3)
    e = a.fmt_b == FP8_E4M3 ? launch_fmt<FP8_E4M3, FP8_E4M3>(a, sms, st) : launch_fmt<FP8_E4M3, FP8_E5M2>(a, sms, st);
  else
    e = a.fmt_b == FP8_E4M3 ? launch_fmt<FP8_E5M2, FP8_E4M3>(a, sms, st) : launch_fmt<FP8_E5M2, FP8_E5M2>(a, sms, st);
  return e == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

}  // namespace fp8ds
