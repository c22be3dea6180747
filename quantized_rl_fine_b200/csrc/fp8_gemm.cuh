// Host-side interface of the grouped FP8 GEMM (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moeq {

struct Fp8GemmArgs {
  const int32_t* offsets;      // [E+1] expert row offsets
  const int32_t* active;       // [E] active experts (ascending)
  const int32_t* num_active;   // [1]
  int32_t E, N, K;             // weight stack dims, W[e] is [N][K]
  int32_t M;                   // rows
  int32_t R;                   // reduction length (forward: K; backward: N)
  int32_t n_ftiles;            // feature tiles per expert
  int32_t nkb, NB, KB;         // 128-wide blocks of R, N and K
  const float* a_scales;       // [ceil(R/128)][M]
  const float* w_scales;       // [E][ceil(N/128)][ceil(K/128)]
  uint8_t* out;                // bf16 [M][F], or e4m3 rows (SwiGLU epilogues)
  float* out_scales;           // e4m3 rows: [blocks][M]
  uint8_t* saved;              // checkpoint e4m3 [M][2f]: written (forward, may be NULL) or read
  uint8_t* saved_scales;       // checkpoint E8M0 [2f/32][M]
  int32_t w_once;              // 1: weights leave L2 first (few rows an expert)
};

// form: 0 single CTAs on 128 token rows, 1 clusters of two CTAs on 256 (grid: CTAs,
// even), 2 and 3 single CTAs on 32 and 64. The row map's box has 128, 128, 32, 64 rows.
cudaError_t launch_grouped_fp8_gemm(bool bwd, int epi, const CUtensorMap& ta, const CUtensorMap& tw,
                                    const Fp8GemmArgs& p, int form, int grid, cudaStream_t s);

}  // namespace moeq
