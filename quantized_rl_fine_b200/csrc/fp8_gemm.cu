// Grouped product of FP8 rows with FP8 expert weights, scales per block of 128
// (forward and dX backward, plain and SwiGLU epilogues).
//
//   forward   acc[p][n] = sum_b sa[b][p] sw[n/128][b] sum_{k in b} a[p][k] W[e][n][k]
//   backward  acc[p][k] = sum_b sd[b][p] sw[b][k/128] sum_{n in b} d[p][n] W[e][n][k]
//
// A tile is 128 token rows (MMA M, one tensor-memory lane each) x 256 output
// features (MMA N). Each 128-long block of the reduction is four
// tcgen05.mma kind::f8f6f4 (K = 32) into one of two tensor-memory buffers of
// 256 columns; eight epilogue warps read the finished buffer and add it, times
// the row's and the weight block's scale, to FP32 accumulators in registers
// while the tensor core fills the other buffer. With a lane per token the
// scale is one number a thread and block, and a row's 128-wide output blocks
// lie inside one thread, which the quantizing epilogues use.
//
// What bounds it: the weight stream below about 340 rows an expert (a block of
// 256 x 128 weights is 32 KiB; at 6.5 TB/s over 148 SMs that is 1.4 us, the four
// MMAs take 0.3), the FP8 tensor rate above. 128 rows a tile waste MMA rows for small
// experts, which costs nothing while the stream is the bound.
//
// The backward reads the same weights in place, as the MN-major B operand:
// features contiguous, 128-byte swizzled blocks of 128 features.
//
// Every wait is bounded; on a timeout the kernel records a device error, lets
// its copies and MMAs in flight finish (again bounded), frees tensor memory
// and returns.
#include <algorithm>

#include "fp8.cuh"
#include "fp8_gemm.cuh"

namespace moeq {

namespace {

constexpr int kRows8 = 128;              // token rows per tile (MMA M)
constexpr int kBox8 = 128;               // one weight box: 128 rows x 128 bytes
constexpr uint32_t kBoxBytes = 16384;
constexpr uint32_t kStage8 = 3 * kBoxBytes;
constexpr int kStages8 = 4;
constexpr int kEpiWarps8 = 8;
constexpr int kThreads8 = 32 * (2 + kEpiWarps8);

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 in, FP32 accumulation, K = 32.
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4: FP32 D, e4m3 A and B (format 0).
__host__ __device__ constexpr uint32_t idesc_f8(uint32_t M, uint32_t N, uint32_t b_mn) {
  return (1u << 4) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

struct Tile8 {
  int e, ft, row0, row_end;
};

// Tile t: feature tile major, token tile minor inside an expert, experts in
// active order, so the tiles in flight share weights first.
__device__ __forceinline__ Tile8 tile8_at(const Fp8GemmArgs& p, const int32_t* tile_start, int A, int t) {
  int lo = 0, hi = A - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile_start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  Tile8 r;
  r.e = p.active[lo];
  const int seg0 = p.offsets[r.e], seg1 = p.offsets[r.e + 1];
  const int nrt = (seg1 - seg0 + kRows8 - 1) / kRows8;
  const int local = t - tile_start[lo];
  r.ft = local / nrt;
  r.row0 = seg0 + (local - r.ft * nrt) * kRows8;
  r.row_end = min(seg1, r.row0 + kRows8);
  return r;
}

// tile_start[a]: tiles of the active experts before a; tile_start[A]: all.
// Tables that do not describe M rows (or name an expert outside the stack)
// give an empty list and the device error.
__device__ int build_tiles8(const Fp8GemmArgs& p, int32_t* tile_start, int32_t* warp_tot) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, nw = blockDim.x >> 5;
  const int A_raw = *p.num_active;
  const bool shape_ok = A_raw >= 0 && A_raw <= p.E && p.offsets[0] == 0 && p.offsets[p.E] == p.M;
  const int A = shape_ok ? A_raw : 0;
  const int per = (A + blockDim.x - 1) / blockDim.x;
  const int a0 = min(A, tid * per), a1 = min(A, a0 + per);
  int local = 0;
  bool bad = !shape_ok;
  for (int a = a0; a < a1; ++a) {
    const int e = p.active[a];
    if (e < 0 || e >= p.E) { bad = true; continue; }
    const int m = p.offsets[e + 1] - p.offsets[e];
    if (m < 0 || m > p.M) { bad = true; continue; }
    local += p.n_ftiles * ((m + kRows8 - 1) / kRows8);
  }
  if (__syncthreads_or(bad ? 1 : 0)) {
    if (tid == 0) {
      if (blockIdx.x == 0) raise_device_error(MOE_DEVERR_BAD_OFFSETS);
      tile_start[0] = 0;
    }
    __syncthreads();
    return 0;
  }
  int x = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_tot[w] = x;
  __syncthreads();
  int run = x - local;
  for (int i = 0; i < w; ++i) run += warp_tot[i];
  for (int a = a0; a < a1; ++a) {
    tile_start[a] = run;
    const int e = p.active[a];
    run += p.n_ftiles * ((p.offsets[e + 1] - p.offsets[e] + kRows8 - 1) / kRows8);
  }
  if (tid == 0) {
    int total = 0;
    for (int i = 0; i < nw; ++i) total += warp_tot[i];
    tile_start[A] = total;
  }
  __syncthreads();
  return A;
}

// 32 bytes to global memory, 16-byte aligned.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&v)[8]) {
  uint4* d = static_cast<uint4*>(dst);
  d[0] = make_uint4(v[0], v[1], v[2], v[3]);
  d[1] = make_uint4(v[4], v[5], v[6], v[7]);
}

// 32 floats times inv as 32 e4m3 bytes.
__device__ __forceinline__ void quantize32(const float* f, float inv, uint8_t* dst) {
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o[i] = cvt_e4m3x4(inf_to_nan(f[4 * i]) * inv, inf_to_nan(f[4 * i + 1]) * inv,
                      inf_to_nan(f[4 * i + 2]) * inv, inf_to_nan(f[4 * i + 3]) * inv);
  store32(dst, o);
}

template <int BWD, int EPI>
__global__ void __launch_bounds__(kThreads8, 1)
grouped_fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm_a,
                        const __grid_constant__ CUtensorMap tm_w, const Fp8GemmArgs p) {
  constexpr bool kGlu = !BWD && EPI == MOE_EPI_SWIGLU;
  constexpr bool kGluBwd = BWD && EPI == MOE_EPI_SWIGLU_BWD;
  extern __shared__ uint8_t smem_raw8[];
  const uint32_t raw = smem_u32(smem_raw8);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw8 + (base - raw);
  constexpr int S = kStages8;
  auto A_at = [&](int s) { return base + s * kStage8; };
  auto B_at = [&](int s) { return base + s * kStage8 + kBoxBytes; };
  const uint32_t bars = base + S * kStage8;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (S + s); };
  auto acc_full = [&](int b) { return bars + 8u * (2 * S + b); };
  auto acc_empty = [&](int b) { return bars + 8u * (2 * S + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (2 * S + 4);
  const uint32_t amax_bar = bars + 8u * (2 * S + 5);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + S * kStage8 + 8u * (2 * S + 6));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* row_amax = reinterpret_cast<float*>(tmem_slot + 2);                 // [2 tiles][2][128]
  int32_t* warp_tot = reinterpret_cast<int32_t*>(row_amax + 4 * kRows8);     // [32]
  int32_t* tile_start = warp_tot + 32;                                       // [E + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), kEpiWarps8);
    }
    mbar_init(drain_bar, 1);
    mbar_init(amax_bar, kEpiWarps8);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_w);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();

  const int A = build_tiles8(p, tile_start, warp_tot);
  const int total = tile_start[A];
  const int nkb = (p.R + 127) / 128;      // blocks of the reduction
  const int f_half = p.N >> 1;            // SwiGLU: first up row

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_a = l2_policy_evict_last();
      const uint64_t pol_w = l2_policy_evict_first();
      int st = 0;
      uint32_t ph = 0;
      long long issued = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const Tile8 tl = tile8_at(p, tile_start, A, t);
        const int c0 = kGlu ? tl.ft * 128 : tl.ft * 256;       // features of the two boxes
        const int c1 = kGlu ? f_half + tl.ft * 128 : c0 + 128;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(empty(st), ph ^ 1u, abort_flag)) { ok = false; break; }
          const uint32_t bar = full(st);
          mbar_arrive_expect_tx(bar, kStage8);
          tma_load_3d_hint(A_at(st), &tm_a, bar, kb * 128, tl.row0, 0, pol_a);
          if constexpr (BWD) {
            tma_load_3d_hint(B_at(st), &tm_w, bar, c0, kb * 128, tl.e, pol_w);
            tma_load_3d_hint(B_at(st) + kBoxBytes, &tm_w, bar, c1, kb * 128, tl.e, pol_w);
          } else {
            tma_load_3d_hint(B_at(st), &tm_w, bar, kb * 128, c0, tl.e, pol_w);
            tma_load_3d_hint(B_at(st) + kBoxBytes, &tm_w, bar, kb * 128, c1, tl.e, pol_w);
          }
          ++issued;
          if (++st == S) { st = 0; ph ^= 1u; }
        }
      }
      if (!ok) {
        // copies in flight land before the CTA can exit
        for (long long g = issued > S ? issued - S : 0; g < issued; ++g)
          mbar_drain(full(static_cast<int>(g % S)), static_cast<uint32_t>((g / S) & 1));
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc = idesc_f8(kRows8, 256, BWD ? 1u : 0u);
    int st = 0;
    uint32_t ph = 0;
    long long it = 0;                     // reduction blocks handed over (buffer it % 2)
    bool ok = true;
    auto wait_w = [&](uint32_t bar, uint32_t parity) {
      const bool r = mbar_wait(bar, parity, abort_flag);
      return __shfl_sync(0xffffffffu, r ? 1 : 0, 0) != 0;
    };
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const int b = static_cast<int>(it & 1);
        if (!wait_w(acc_empty(b), static_cast<uint32_t>((it >> 1) & 1) ^ 1u)) { ok = false; break; }
        if (!wait_w(full(st), ph)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d = tmem_base + static_cast<uint32_t>(b) * 256u;
          const uint64_t da = smem_desc_sw128(A_at(st), 16, 1024);
          const uint64_t db = BWD ? smem_desc_sw128(B_at(st), kBoxBytes, 1024)
                                  : smem_desc_sw128(B_at(st), 16, 1024);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)   // 32 of the 128 reduction elements each
            mma_f8_ss(d, da + 2 * ks, db + (BWD ? 256 : 2) * ks, idesc, ks > 0 ? 1u : 0u);
          mma_commit(empty(st));
          mma_commit(acc_full(b));
        }
        __syncwarp();
        if (++st == S) { st = 0; ph ^= 1u; }
      }
    }
    if (elect_one()) mma_commit(drain_bar);
    __syncwarp();
    if (lane == 0) mbar_drain(drain_bar, 0);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ scaled sum and epilogue
    const int q = warp & 3;                      // tensor-memory lane quarter
    const int wg = (warp - 2) >> 2;              // column half
    const int r_in = q * 32 + lane;              // row of the tile
    const uint32_t tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    // This thread's 128 columns: plain, the half's box; SwiGLU, 64 gate
    // columns and the 64 matching up columns.
    const uint32_t col0 = kGlu ? static_cast<uint32_t>(wg * 64) : static_cast<uint32_t>(wg * 128);
    const uint32_t col1 = kGlu ? 128u + static_cast<uint32_t>(wg * 64) : col0 + 64u;
    const int KB = (p.K + 127) / 128, NB = (p.N + 127) / 128;
    long long it = 0;
    bool ok = true;
    int li = 0;                                  // this CTA's tile count
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x, ++li) {
      const Tile8 tl = tile8_at(p, tile_start, A, t);
      const int row = tl.row0 + r_in;
      const bool row_ok = row < tl.row_end;
      const float* sa = p.a_scales + min(row, p.M - 1);
      const float* swe = p.w_scales + static_cast<int64_t>(tl.e) * NB * KB;
      // Weight scales of this thread's two 64-column halves, one per reduction
      // block: sw0[kb * step], sw1[kb * step]. Blocks past the last feature
      // (a tile that ends early) are clamped; their columns are not stored.
      int b0, b1;
      if constexpr (kGlu) { b0 = tl.ft; b1 = f_half / 128 + tl.ft; }
      else { b0 = b1 = min(tl.ft * 2 + wg, (BWD ? KB : NB) - 1); }
      const float* sw0 = BWD ? swe + b0 : swe + static_cast<int64_t>(b0) * KB;
      const float* sw1 = BWD ? swe + b1 : swe + static_cast<int64_t>(b1) * KB;
      const int step = BWD ? KB : 1;
      float acc[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
      float na = __ldg(sa), n0 = __ldg(sw0), n1 = kGlu ? __ldg(sw1) : 0.0f;
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const float s0 = na * n0, s1 = kGlu ? na * n1 : s0;
        if (kb + 1 < nkb) {
          na = __ldg(sa + static_cast<int64_t>(kb + 1) * p.M);
          n0 = __ldg(sw0 + (kb + 1) * step);
          if constexpr (kGlu) n1 = __ldg(sw1 + (kb + 1) * step);
        }
        const int b = static_cast<int>(it & 1);
        const bool r = mbar_wait(acc_full(b), static_cast<uint32_t>((it >> 1) & 1), abort_flag);
        if (!__shfl_sync(0xffffffffu, r ? 1 : 0, 0)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tb = tq + static_cast<uint32_t>(b) * 256u;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tb + (c < 2 ? col0 : col1) + 32u * (c & 1), v);
          tmem_wait_ld();
          const float s = c < 2 ? s0 : s1;
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[32 * c + j] = fmaf(s, __uint_as_float(v[j]), acc[32 * c + j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(b));
      }
      if (!ok) break;

      if constexpr (kGlu) {
        // acc[0..63] gate, acc[64..127] up of features f0 ..
        const int f0 = tl.ft * 128 + wg * 64;
        if (p.saved != nullptr && row_ok) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j) m = fmaxf(m, finite_abs(acc[32 * c + j]));
            const int e = fp8_block_exp(m);
            const int col = (c < 2 ? f0 : f_half + f0) + 32 * (c & 1);
            quantize32(acc + 32 * c, exp2_int(-e), p.saved + static_cast<int64_t>(row) * p.N + col);
            p.saved_scales[static_cast<int64_t>(col / 32) * p.M + row] = static_cast<uint8_t>(e + 127);
          }
        }
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 64; ++j) {
          acc[j] = silu_f(acc[j]) * acc[64 + j];
          m = fmaxf(m, finite_abs(acc[j]));
        }
        // The block of 128 features spans both column halves. Two exchange
        // buffers in turn: passing tile n + 1's barrier means that everybody
        // has read tile n's, which tile n + 2 then writes.
        float* xch = row_amax + (li & 1) * 2 * kRows8;
        xch[wg * kRows8 + r_in] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(amax_bar);
        const bool met = mbar_wait(amax_bar, static_cast<uint32_t>(li & 1), abort_flag);
        if (!__shfl_sync(0xffffffffu, met ? 1 : 0, 0)) break;
        m = fmaxf(m, xch[(wg ^ 1) * kRows8 + r_in]);
        if (row_ok) {
          const int e = fp8_block_exp(m);
          const float inv = exp2_int(-e);
          uint8_t* dst = p.out + static_cast<int64_t>(row) * f_half + f0;
          quantize32(acc, inv, dst);
          quantize32(acc + 32, inv, dst + 32);
          if (wg == 0) p.out_scales[static_cast<int64_t>(tl.ft) * p.M + row] = exp2_int(e);
        }
      } else if constexpr (kGluBwd) {
        const int f0 = tl.ft * 256 + wg * 128;       // features f0 .. f0 + 127 of dh
        const int K = p.K;
        if (row_ok && f0 < K) {
          const uint8_t* gq = p.saved + static_cast<int64_t>(row) * (2 * K) + f0;
          float mg = 0.0f, mu = 0.0f;
          // acc[2i], acc[2i+1] (dh of a feature pair) become the BF16 pairs dg, du.
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int64_t grp = f0 / 32 + c;
            const int xg = p.saved_scales[grp * p.M + row];
            const int xu = p.saved_scales[(grp + K / 32) * p.M + row];
            const float sg = e8m0_to_float(xg), su = e8m0_to_float(xu);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 g4 = __ldg(reinterpret_cast<const uint4*>(gq + 32 * c + 16 * h));
              const uint4 u4 = __ldg(reinterpret_cast<const uint4*>(gq + K + 32 * c + 16 * h));
              const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 g2 = e4m3x2_to_float2(gw[i >> 1] >> (16 * (i & 1)));
                const float2 u2 = e4m3x2_to_float2(uw[i >> 1] >> (16 * (i & 1)));
                const int a = 32 * c + 16 * h + 2 * i;
                float dg[2], du[2];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const float g = (z ? g2.y : g2.x) * sg, u = (z ? u2.y : u2.x) * su;
                  const float s = sigmoid_f(g), x = acc[a + z];
                  dg[z] = x * u * s * (1.0f + g * (1.0f - s));
                  du[z] = x * g * s;
                }
                const uint32_t pg = pack_bf16x2(dg[0], dg[1]), pu = pack_bf16x2(du[0], du[1]);
                mg = fmaxf(mg, fmaxf(finite_abs(bf16_bits_to_float(pg & 0xffffu)),
                                     finite_abs(__uint_as_float(pg & 0xffff0000u))));
                mu = fmaxf(mu, fmaxf(finite_abs(bf16_bits_to_float(pu & 0xffffu)),
                                     finite_abs(__uint_as_float(pu & 0xffff0000u))));
                acc[a] = __uint_as_float(pg);
                acc[a + 1] = __uint_as_float(pu);
              }
            }
          }
          const int eg = fp8_block_exp(mg), eu = fp8_block_exp(mu);
          uint8_t* dst = p.out + static_cast<int64_t>(row) * (2 * K) + f0;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float inv = exp2_int(half ? -eu : -eg);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float f[32];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint32_t w = __float_as_uint(acc[32 * c + 2 * i + half]);
                f[2 * i] = bf16_bits_to_float(w & 0xffffu);
                f[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
              }
              quantize32(f, inv, dst + half * K + 32 * c);
            }
          }
          const int64_t blk = f0 / 128;
          p.out_scales[blk * p.M + row] = exp2_int(eg);
          p.out_scales[(blk + K / 128) * p.M + row] = exp2_int(eu);
        }
      } else {
        const int F = BWD ? p.K : p.N;
        const int f0 = tl.ft * 256 + wg * 128;
        if (row_ok) {
          uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + static_cast<int64_t>(row) * F + f0;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (f0 + 16 * c >= F) break;             // F % 16 == 0
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = pack_bf16x2(acc[16 * c + 2 * i], acc[16 * c + 2 * i + 1]);
            store32(dst + 16 * c, o);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, 512);
}

}  // namespace

cudaError_t launch_grouped_fp8_gemm(bool bwd, int epi, const CUtensorMap& ta, const CUtensorMap& tw,
                                    const Fp8GemmArgs& p, int grid, cudaStream_t s) {
  const size_t smem = 1024 + kStages8 * kStage8 + 8 * (2 * kStages8 + 6) + 8 + 4 * 4 * kRows8 + 4 * 32 +
                      4 * (static_cast<size_t>(p.E) + 1);
  auto go = [&](auto kern) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(kThreads8), smem, s, ta, tw, p);
  };
  if (!bwd) return epi == MOE_EPI_SWIGLU ? go(grouped_fp8_gemm_kernel<0, MOE_EPI_SWIGLU>)
                                         : go(grouped_fp8_gemm_kernel<0, MOE_EPI_NONE>);
  return epi == MOE_EPI_SWIGLU_BWD ? go(grouped_fp8_gemm_kernel<1, MOE_EPI_SWIGLU_BWD>)
                                   : go(grouped_fp8_gemm_kernel<1, MOE_EPI_NONE>);
}

}  // namespace moeq
