// Unpermute + gate-weighted combine of the per-slot rows, and its backward
// (gate-scaled scatter of the upstream gradient to the per-slot rows).
// The gates are applied here rather than inside the GEMM epilogue.
//
// One warp per token; each lane moves 16-byte slices (8 BF16) of the rows,
// so every row access is a fully coalesced 512-byte warp transaction.
#include <algorithm>

#include "launchers.cuh"
#include "common.cuh"

namespace moeq {

namespace {

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// BF16 nearest-even of the exact product g * x (x a BF16 value). The FP32
// product can land exactly on a BF16 halfway point while the exact product
// does not; the FMA residual decides that case, so the result has one rounding.
__device__ __forceinline__ uint32_t bf16_of_product(float g, float x) {
  float p = g * x;
  const uint32_t pb = __float_as_uint(p);
  if ((pb & 0xFFFFu) == 0x8000u) {
    const float r = fmaf(g, x, -p);
    if (r != 0.0f) {
      const bool up = (r > 0.0f) == (p > 0.0f);   // exact magnitude above |p|
      p = __uint_as_float(up ? pb + 1u : pb - 1u);
    }
  }
  return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(p)));
}

__global__ void combine_kernel(const uint4* __restrict__ rows, const int32_t* __restrict__ inv_perm,
                               const float* __restrict__ gates, int T, int k, int64_t dvec,
                               uint4* __restrict__ out) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= T) return;
  int32_t idx[32];
  float g[32];
  for (int j = 0; j < k; ++j) {
    idx[j] = inv_perm[static_cast<int64_t>(t) * k + j];
    g[j] = gates ? gates[static_cast<int64_t>(t) * k + j] : 1.0f;
  }
  for (int64_t c = lane; c < dvec; c += 32) {
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j = 0; j < k; ++j) {
      float f[8];
      unpack8(rows[static_cast<int64_t>(idx[j]) * dvec + c], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(g[j], f[i], acc[i]);
    }
    uint4 o;
    o.x = pack_bf16x2(acc[0], acc[1]);
    o.y = pack_bf16x2(acc[2], acc[3]);
    o.z = pack_bf16x2(acc[4], acc[5]);
    o.w = pack_bf16x2(acc[6], acc[7]);
    out[static_cast<int64_t>(t) * dvec + c] = o;
  }
}

__global__ void scatter_kernel(const uint4* __restrict__ rows, const int32_t* __restrict__ inv_perm,
                               const float* __restrict__ gates, int T, int k, int64_t dvec,
                               uint4* __restrict__ out) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= T) return;
  for (int j = 0; j < k; ++j) {
    const int64_t p = inv_perm[static_cast<int64_t>(t) * k + j];
    const float g = gates ? gates[static_cast<int64_t>(t) * k + j] : 1.0f;
    for (int64_t c = lane; c < dvec; c += 32) {
      float f[8];
      unpack8(rows[static_cast<int64_t>(t) * dvec + c], f);
      uint32_t h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = bf16_of_product(g, f[i]);
      uint4 o;
      o.x = h[0] | (h[1] << 16);
      o.y = h[2] | (h[3] << 16);
      o.z = h[4] | (h[5] << 16);
      o.w = h[6] | (h[7] << 16);
      out[p * dvec + c] = o;
    }
  }
}

// bf16_of_product of eight values at once: the halfway case, one product in
// 65536, is looked for in all eight together.
__device__ __forceinline__ uint4 bf16_of_products8(float g, const float (&x)[8]) {
  float p[8];
  uint32_t nearest = 0xffffffffu;          // smallest distance of a product's low half from 0x8000
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = g * x[i];
    nearest = min(nearest, (__float_as_uint(p[i]) & 0xFFFFu) ^ 0x8000u);
  }
  if (nearest == 0u) {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = bf16_of_product(g, x[i]);
    return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
  }
  return make_uint4(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]),
                    pack_bf16x2(p[6], p[7]));
}

// One block per token, 16-byte slices of the row over its threads: dy is read
// once, each of the token's k rows once, and gate * dy written once to each of
// the k slots (bf16_of_product: one rounding, the bits of scatter_kernel). The
// k dot products accumulate in FP32 per thread in ascending slice order, then
// over lanes and warps in a fixed order. Bound: DRAM, 2TD + 2TkD bytes read and
// 2TkD written; 4096 tokens x 8 x 7168 (1.0 GB) take 173 us, 5.8 TB/s. One pass
// with all k rows in flight, so that dy is not read again for the dot products.
template <int KMAX>
__global__ void __launch_bounds__(256)
combine_bwd_kernel(const uint4* __restrict__ dy, const uint4* __restrict__ rows,
                   const int32_t* __restrict__ inv_perm, const float* __restrict__ gates, int k,
                   int64_t dvec, uint4* __restrict__ d_rows, float* __restrict__ d_gates) {
  grid_dependency_wait();
  grid_dependents_launch();
  __shared__ float part[8][KMAX];
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
  int64_t base[KMAX];
  float g[KMAX], acc[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    const int p = (j < k) ? __ldg(inv_perm + t * k + j) : -1;
    base[j] = (p >= 0 && p < static_cast<int>(gridDim.x) * k) ? p * dvec : -1;
    g[j] = (j < k && gates) ? __ldg(gates + t * k + j) : 1.0f;
    acc[j] = 0.0f;
  }
  for (int64_t c = threadIdx.x; c < dvec; c += blockDim.x) {
    uint4 r[KMAX];
    const uint4 dv = __ldcs(dy + t * dvec + c);
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
      if (base[j] >= 0) r[j] = __ldcs(rows + base[j] + c);
    float f[8];
    unpack8(dv, f);
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      if (base[j] < 0) continue;
      float y[8];
      unpack8(r[j], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[j] = fmaf(f[i], y[i], acc[j]);
      __stcs(d_rows + base[j] + c, bf16_of_products8(g[j], f));
    }
  }
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    if (j >= k) continue;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    if (lane == 0) part[warp][j] = acc[j];
  }
  __syncthreads();
  for (int j = threadIdx.x; j < k; j += blockDim.x) {
    float s = 0.0f;
    for (int w = 0; w < nwarps; ++w) s += part[w][j];
    d_gates[t * k + j] = s;
  }
}

}  // namespace

cudaError_t launch_combine_bwd(const void* dy, const void* rows, const int32_t* inv_perm,
                               const float* gates, int T, int k, int64_t D, void* d_rows,
                               float* d_gates, cudaStream_t s) {
  const int64_t dvec = D / 8;
  const int threads = static_cast<int>(std::min<int64_t>(256, (dvec + 31) / 32 * 32));
#define MOEQ_CB(K_)                                                                                 \
  launch_pdl(combine_bwd_kernel<K_>, dim3(T), dim3(threads), 0, s, static_cast<const uint4*>(dy),   \
             static_cast<const uint4*>(rows), inv_perm, gates, k, dvec, static_cast<uint4*>(d_rows), \
             d_gates)
  if (k <= 2) return MOEQ_CB(2);
  if (k <= 4) return MOEQ_CB(4);
  if (k <= 8) return MOEQ_CB(8);
  if (k <= 16) return MOEQ_CB(16);
  return MOEQ_CB(32);
#undef MOEQ_CB
}

cudaError_t launch_combine(const void* rows, const int32_t* inv_perm, const float* gates, int T,
                           int k, int64_t D, void* out, int mode, cudaStream_t s) {
  const int warps = 8;
  const int blocks = (T + warps - 1) / warps;
  return launch_pdl(mode == 0 ? combine_kernel : scatter_kernel, dim3(blocks), dim3(warps * 32), 0,
                    s, static_cast<const uint4*>(rows), inv_perm, gates, T, k, D / 8,
                    static_cast<uint4*>(out));
}

}  // namespace moeq
