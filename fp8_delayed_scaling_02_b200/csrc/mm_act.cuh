// What fp8_mm_act hands to the kernel for a few rows of A.
#pragma once

#include "amax_fold.cuh"
#include "common.cuh"

namespace fp8ds {

struct SkinnyArgs {
  const uint8_t* A;  // [M, K] codes
  const uint8_t* B;  // [N, K] codes
  int M, N, K;
  int fmt_a, fmt_b;
  const float* sinv_a;
  int a_rows;
  const float* sinv_b;
  const float* bias;
  int act;
  const uint16_t* aux;
  int aux_mul;
  uint16_t* z;
  uint16_t* out;     // bf16, or null
  uint8_t* out8;     // codes, with ring and out_fmt
  int out_fmt;
  RingArgs ring;
};

constexpr int kSkinnyMaxM = 32;

bool skinny_wins(int64_t M, int64_t N, int64_t K, int sms);
int launch_skinny(const SkinnyArgs& a, int sms, cudaStream_t st);  // 1 <= M <= kSkinnyMaxM

}  // namespace fp8ds
