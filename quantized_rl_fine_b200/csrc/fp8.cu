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

// Sixteen BF16 values (two 16-byte pieces) of a 128-element block to e4m3; the
// block's eight threads find its largest magnitude with three shuffles.
__device__ __forceinline__ uint4 quantize16(const uint4& a, const uint4& b, float* scale) {
  float f[16];
  bf16x16(a, b, f);
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(f[j]));     // (NaN is passed over)
  if (!(amax < INFINITY)) {                                          // rare
    amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = fmaxf(amax, finite_abs(f[j]));
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] = inf_to_nan(f[j]);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int e = fp8_block_exp(amax);
  const float inv = exp2_int(-e);
  *scale = exp2_int(e);
  return make_uint4(cvt_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                    cvt_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv),
                    cvt_e4m3x4(f[8] * inv, f[9] * inv, f[10] * inv, f[11] * inv),
                    cvt_e4m3x4(f[12] * inv, f[13] * inv, f[14] * inv, f[15] * inv));
}

// A group of 8 / TPB warps per token, TPB tokens a block: each thread takes 16
// elements at a time, two such units in flight. The token is read and
// quantized once and written to its k rows (16-byte stores), which costs k
// writes of one byte an element against k reads of two if every permuted row
// were quantized by itself. Bound: DRAM, read once and written k times;
// 32768 x 7168 111 us (6.4 TB/s), 4096 x 7168 to 8 rows 59 us (5.1 TB/s). Narrower
// rows written to several leave part of a token's 256 threads, which cover 8192
// elements a step, without work: 8192 x 4096 to 8 rows 66 us (5.2 TB/s), 8192 x 2048
// 42.5 (4.0), 16384 x 1024 70 (2.5), all of 26 to 52 us at the copy rate.
template <int TPB>
__global__ void __launch_bounds__(256)
quantize_fp8_kernel(const uint4* __restrict__ x, int T, int64_t K, const int32_t* __restrict__ inv_perm,
                    int k, int M, uint8_t* __restrict__ q, float* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  constexpr int kLanes = 256 / TPB;                           // threads of a token
  const int64_t t = static_cast<int64_t>(blockIdx.x) * TPB + threadIdx.x / kLanes;
  if (t >= T) return;                                         // whole warps
  const int th = threadIdx.x % kLanes, lane = threadIdx.x & 31;
  // Lane j < k holds the token's j-th row (-1: not a row).
  int my_row = -1;
  if (lane < k) {
    my_row = inv_perm ? __ldg(inv_perm + t * k + lane) : static_cast<int>(t);
    if (my_row < 0 || my_row >= M) my_row = -1;
  }
  const int units = static_cast<int>(K / 16);
  const uint4* src = x + t * (K / 8);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int base = 0; base < units; base += 2 * kLanes) {      // uniform over the warp: every lane shuffles
    uint4 v[2][2], o[2];
    float sc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int un = base + i * kLanes + th;
      v[i][0] = un < units ? __ldcs(src + 2 * un) : zero;
      v[i][1] = un < units ? __ldcs(src + 2 * un + 1) : zero;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) o[i] = quantize16(v[i][0], v[i][1], &sc[i]);
    for (int j = 0; j < k; ++j) {
      const int64_t r = __shfl_sync(0xffffffffu, my_row, j);
      if (r < 0) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int un = base + i * kLanes + th;
        if (un >= units) continue;
        *reinterpret_cast<uint4*>(q + r * K + 16ll * un) = o[i];
        if ((un & 7) == 0) scales[static_cast<int64_t>(un >> 3) * M + r] = sc[i];
      }
    }
  }
}

// BF16 of the exact product of an e4m3 value and any FP32 scale, rounded once.
// It has up to 28 bits; their rounding to FP32 can end on a halfway point
// between two BF16 values, and then the exact product (in 64 bits) decides.
__device__ __forceinline__ uint32_t bf16_of_scaled(float q, float s) {
  float p = q * s;
  const uint32_t b = __float_as_uint(p);
  if ((b & 0xffffu) == 0x8000u) {
    const double rest = static_cast<double>(q) * s - p;
    if (rest != 0.0) p = __uint_as_float((rest > 0.0) == (p > 0.0f) ? b + 1u : b - 1u);
  }
  return pack_bf16x2(p, 0.0f);
}

// Eight of them; the halfway points are looked for in all eight together.
__device__ __forceinline__ uint4 bf16_of_scaled8(const float (&q)[8], float s) {
  float p[8];
  uint32_t nearest = 0xffffffffu;             // smallest distance of a product's low half from 0x8000
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = q[i] * s;
    nearest = min(nearest, (__float_as_uint(p[i]) & 0xffffu) ^ 0x8000u);
  }
  if (nearest == 0u) {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = bf16_of_scaled(q[i], s);
    return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
  }
  return make_uint4(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]), pack_bf16x2(p[6], p[7]));
}

// Blocks of 8 rows x 1024 elements, one row a warp: the rows' scales of a block
// column lie next to each other and share their memory sectors. Eight elements
// a lane and step, so that both the loads (8 bytes) and the stores (16) of a
// warp are contiguous: 16 elements a lane, two stores 32 bytes apart, wrote
// every sector in halves (32768 x 4096: 83 us). Bound: DRAM; 32768 x 4096 with
// 1 x 32 blocks 66 us, 6.2 TB/s, and the same with FP32 scales (64 without the
// look for halfway points).
template <int FMT>
__global__ void __launch_bounds__(256)
dequantize_fp8_kernel(const uint8_t* __restrict__ q, const void* __restrict__ scales, int M, int64_t K,
                      uint16_t* __restrict__ out) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t m = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int units = static_cast<int>(K / 8);
  if (m >= M) return;
  for (int base = blockIdx.y * 128; base < units; base += 128 * gridDim.y) {
    uint2 v[4];
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int un = base + 32 * i + lane;
      if (un >= units) continue;
      v[i] = __ldcs(reinterpret_cast<const uint2*>(q + m * K) + un);
      if constexpr (FMT == MOE_FP8_BLOCK128_F32)
        s[i] = __ldg(static_cast<const float*>(scales) + static_cast<int64_t>(un >> 4) * M + m);
      else
        s[i] = e8m0_to_float(__ldg(static_cast<const uint8_t*>(scales) + static_cast<int64_t>(un >> 2) * M + m));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int un = base + 32 * i + lane;
      if (un >= units) continue;
      const float2 a = e4m3x2_to_float2(v[i].x), b = e4m3x2_to_float2(v[i].x >> 16);
      const float2 c = e4m3x2_to_float2(v[i].y), d = e4m3x2_to_float2(v[i].y >> 16);
      uint4 o;
      if constexpr (FMT == MOE_FP8_BLOCK128_F32) {
        const float f[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
        o = bf16_of_scaled8(f, s[i]);
      } else {                                // (a power of two: the FP32 product is exact)
        o = make_uint4(pack_bf16x2(a.x * s[i], a.y * s[i]), pack_bf16x2(b.x * s[i], b.y * s[i]),
                       pack_bf16x2(c.x * s[i], c.y * s[i]), pack_bf16x2(d.x * s[i], d.y * s[i]));
      }
      __stcs(reinterpret_cast<uint4*>(out + m * K) + un, o);
    }
  }
}

}  // namespace

cudaError_t launch_quantize_fp8_rows(const void* x, int T, int64_t K, const int32_t* inv_perm, int k,
                                     void* q, float* scales, cudaStream_t s) {
  // A warp per token when there are enough tokens to fill the SMs that way and
  // each is written once (32768 x 7168: 112 us, 150 with a block per token);
  // a block per token for few tokens (latency), and when a token is written to
  // k rows (4096 x 7168 to 8 rows: 59 us, some 20 more with a warp per token). The
  // latter is measured at K = 7168 only.
  const int tpb = K <= 512 || (T >= 4096 && k == 1) ? 8 : 1;
  auto kern = tpb == 8 ? quantize_fp8_kernel<8> : quantize_fp8_kernel<1>;
  return launch_pdl(kern, dim3(blocks_for(T, tpb)), dim3(256), 0, s, static_cast<const uint4*>(x), T, K,
                    inv_perm, k, T * k, static_cast<uint8_t*>(q), scales);
}

cudaError_t launch_dequantize_fp8_rows(const void* q, const void* scales, int M, int64_t K, int fmt,
                                       void* out, cudaStream_t s) {
  const int64_t cols = (K / 8 + 127) / 128;
  const dim3 grid(blocks_for(M, 8), static_cast<unsigned>(std::min<int64_t>(cols, 65535)));
  auto kern = fmt == MOE_FP8_BLOCK128_F32 ? dequantize_fp8_kernel<MOE_FP8_BLOCK128_F32>
                                          : dequantize_fp8_kernel<MOE_FP8_BLOCK32_E8M0>;
  return launch_pdl(kern, grid, dim3(256), 0, s, static_cast<const uint8_t*>(q), scales, M, K,
                    static_cast<uint16_t*>(out));
}

}  // namespace moeq
