// BF16 rows to FP8 rows (e4m3, one power-of-two scale per 1 x 128 block) and
// back. Definitions: include/moeq.h, "FP8 rows and weights".
#include <algorithm>

#include "fp8.cuh"
#include "launchers.cuh"

namespace moeq {

namespace {

__device__ __forceinline__ void bf16x16(const uint4& u, const uint4& v, float (&f)[16]) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// One block per token. A thread takes 16 elements (two 16-byte loads); the
// eight threads of a 128-element block find its largest magnitude with three
// shuffles. The token is read and quantized once and written to its k rows
// (16-byte stores), which costs k writes of one byte an element against k
// reads of two if every permuted row were quantized by itself.
__global__ void __launch_bounds__(256)
quantize_fp8_kernel(const uint4* __restrict__ x, int64_t K, const int32_t* __restrict__ inv_perm,
                    int k, int M, uint8_t* __restrict__ q, float* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31;
  // Lane j < k holds the token's j-th row (-1: not a row).
  int my_row = -1;
  if (lane < k) {
    my_row = inv_perm ? __ldg(inv_perm + t * k + lane) : static_cast<int>(t);
    if (my_row < 0 || my_row >= M) my_row = -1;
  }
  const int units = static_cast<int>(K / 16);
  const int steps = (units + blockDim.x - 1) / blockDim.x;    // uniform: every thread shuffles
  for (int i = 0; i < steps; ++i) {
    const int un = i * blockDim.x + threadIdx.x;
    const bool ok = un < units;
    float f[16];
    {
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (ok) {
        const uint4* src = x + t * (K / 8) + 2 * un;
        a = __ldg(src);
        b = __ldg(src + 1);
      }
      bf16x16(a, b, f);
    }
    float amax = 0.0f;
    bool odd = false;                       // holds a value that is not finite
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      amax = fmaxf(amax, finite_abs(f[j]));
      odd |= !(fabsf(f[j]) < INFINITY);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int e = fp8_block_exp(amax);
    const float inv = exp2_int(-e);
    if (odd) {
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = inf_to_nan(f[j]);
    }
    uint4 o;
    o.x = cvt_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    o.y = cvt_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
    o.z = cvt_e4m3x4(f[8] * inv, f[9] * inv, f[10] * inv, f[11] * inv);
    o.w = cvt_e4m3x4(f[12] * inv, f[13] * inv, f[14] * inv, f[15] * inv);
    const float sc = exp2_int(e);
    for (int j = 0; j < k; ++j) {
      const int64_t r = __shfl_sync(0xffffffffu, my_row, j);
      if (!ok || r < 0) continue;
      *reinterpret_cast<uint4*>(q + r * K + 16 * un) = o;
      if ((un & 7) == 0) scales[static_cast<int64_t>(un >> 3) * M + r] = sc;
    }
  }
}

// Blocks of 8 rows x 32 units of 16 elements, one row a warp: the rows' scales
// of a block column lie next to each other and share their memory sectors.
template <int FMT>
__global__ void __launch_bounds__(256)
dequantize_fp8_kernel(const uint8_t* __restrict__ q, const void* __restrict__ scales, int M, int64_t K,
                      uint16_t* __restrict__ out) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t m = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int units = static_cast<int>(K / 16);
  if (m >= M) return;
  for (int un = blockIdx.y * 32 + lane; un < units; un += 32 * gridDim.y) {
    float s;
    if constexpr (FMT == MOE_FP8_BLOCK128_F32) {
      s = __ldg(static_cast<const float*>(scales) + static_cast<int64_t>(un >> 3) * M + m);
    } else {
      const int X = __ldg(static_cast<const uint8_t*>(scales) + static_cast<int64_t>(un >> 1) * M + m);
      s = e8m0_to_float(X);
    }
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(q + m * K) + un);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 lo = e4m3x2_to_float2(w[i]), hi = e4m3x2_to_float2(w[i] >> 16);
      o[2 * i] = pack_bf16x2(lo.x * s, lo.y * s);
      o[2 * i + 1] = pack_bf16x2(hi.x * s, hi.y * s);
    }
    uint4* dst = reinterpret_cast<uint4*>(out + m * K) + 2 * un;
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace

cudaError_t launch_quantize_fp8_rows(const void* x, int T, int64_t K, const int32_t* inv_perm, int k,
                                     void* q, float* scales, cudaStream_t s) {
  const int threads = static_cast<int>(std::min<int64_t>(256, (K / 16 + 31) / 32 * 32));
  return launch_pdl(quantize_fp8_kernel, dim3(T), dim3(threads), 0, s, static_cast<const uint4*>(x), K,
                    inv_perm, k, T * k, static_cast<uint8_t*>(q), scales);
}

cudaError_t launch_dequantize_fp8_rows(const void* q, const void* scales, int M, int64_t K, int fmt,
                                       void* out, cudaStream_t s) {
  const int64_t cols = (K / 16 + 31) / 32;
  const dim3 grid((M + 7) / 8, static_cast<unsigned>(std::min<int64_t>(cols, 65535)));
  auto kern = fmt == MOE_FP8_BLOCK128_F32 ? dequantize_fp8_kernel<MOE_FP8_BLOCK128_F32>
                                          : dequantize_fp8_kernel<MOE_FP8_BLOCK32_E8M0>;
  return launch_pdl(kern, grid, dim3(256), 0, s, static_cast<const uint8_t*>(q), scales, M, K,
                    static_cast<uint16_t*>(out));
}

}  // namespace moeq
