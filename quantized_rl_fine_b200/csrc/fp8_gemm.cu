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
constexpr uint32_t kBoxBytes = 16384;    // one operand box: 128 rows x 128 bytes
constexpr uint32_t kStage8 = 3 * kBoxBytes;
constexpr int kStages8 = 3;
constexpr int kEpiWarp8 = 4;             // warp 0 copies, warp 1 issues MMAs, warps 4-11 epilogue
constexpr int kEpiWarps8 = 8;
constexpr int kThreads8 = 32 * (kEpiWarp8 + kEpiWarps8);
// Registers: 168 a thread at launch (384 x 168 = 64512); the first warpgroup
// gives up 128 a thread and the two epilogue warpgroups take 64 each: 128 x 40
// + 256 x 232 = 64512. An epilogue thread holds 128 accumulators and 64 values in flight.
constexpr int kRegsCopy = 40, kRegsEpi = 232;
static_assert(128 * kRegsCopy + 256 * kRegsEpi <= kThreads8 * 168, "register split");
// Output staging of one epilogue thread: its 256 bytes of a row, padded so
// that the 16-byte stores of eight neighbouring threads fall in distinct banks.
constexpr uint32_t kSlot8 = 272;
constexpr size_t smem_bytes8(int E) {
  return 1024 + kStages8 * kStage8 + 256 * kSlot8 + 8 * (2 * kStages8 + 8) + 16 + 4 * 4 * kRows8 + 4 * 32 +
         4 * 2 * (static_cast<size_t>(E) + 1) + 2 * static_cast<size_t>(E);
}
static_assert(smem_bytes8(1024) <= 227 * 1024, "shared memory of the largest stack");

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

// The tile list in shared memory: for the a-th active expert its first tile,
// its first row and its id; start[A] is the number of tiles, seg[A] = M.
struct TileList8 {
  int32_t* start;
  int32_t* seg;
  uint16_t* id;
  int A;
};

struct Tile8 {
  int e, ft, row0, row_end, a;
};

// Tile t (a0: active index of an earlier tile): feature tile major, token tile
// minor inside an expert, experts in active order, so the tiles in flight
// share weights first.
__device__ __forceinline__ Tile8 tile8_at(const TileList8& tl, int t, int a0) {
  int lo = a0, hi = tl.A - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tl.start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  Tile8 r;
  r.a = lo;
  r.e = tl.id[lo];
  const int seg0 = tl.seg[lo], seg1 = tl.seg[lo + 1];
  const int nrt = (seg1 - seg0 + kRows8 - 1) / kRows8;
  const int local = t - tl.start[lo];
  r.ft = local / nrt;
  r.row0 = seg0 + (local - r.ft * nrt) * kRows8;
  r.row_end = min(seg1, r.row0 + kRows8);
  return r;
}

// Builds the list; the active experts' rows must lie behind one another from
// 0 to M. Tables that do not say so (or name an expert outside the stack) give
// an empty list and the device error.
__device__ void build_tiles8(const Fp8GemmArgs& p, TileList8& tl, int32_t* warp_tot) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, nw = blockDim.x >> 5;
  const int A_raw = *p.num_active;
  bool bad = !(A_raw >= 1 && A_raw <= p.E && p.offsets[0] == 0 && p.offsets[p.E] == p.M);
  const int A = bad ? 0 : A_raw;
  const int per = (A + blockDim.x - 1) / blockDim.x;      // <= 3
  const int a0 = min(A, tid * per), a1 = min(A, a0 + per);
  int local = 0;
  for (int a = a0; a < a1; ++a) {
    const int e = p.active[a];
    if (e < 0 || e >= p.E) { bad = true; continue; }
    const int s0 = p.offsets[e], s1 = p.offsets[e + 1];
    const int en = a + 1 < A ? p.active[a + 1] : p.E;
    if (s0 < 0 || s1 <= s0 || s1 > p.M || (a == 0 && s0 != 0) || en <= e || en > p.E ||
        p.offsets[en] != s1) {
      bad = true;
      continue;
    }
    tl.seg[a] = s0;
    tl.id[a] = static_cast<uint16_t>(e);
    local += p.n_ftiles * ((s1 - s0 + kRows8 - 1) / kRows8);
  }
  if (__syncthreads_or(bad ? 1 : 0)) {
    if (tid == 0) {
      if (blockIdx.x == 0) raise_device_error(MOE_DEVERR_BAD_OFFSETS);
      tl.start[0] = 0;
    }
    tl.A = 0;
    __syncthreads();
    return;
  }
  int x = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_tot[w] = x;
  if (tid == 0) tl.seg[A] = p.M;
  __syncthreads();
  int run = x - local;
  for (int i = 0; i < w; ++i) run += warp_tot[i];
  for (int a = a0; a < a1; ++a) {
    tl.start[a] = run;
    run += p.n_ftiles * ((tl.seg[a + 1] - tl.seg[a] + kRows8 - 1) / kRows8);
  }
  if (tid == 0) {
    int total = 0;
    for (int i = 0; i < nw; ++i) total += warp_tot[i];
    tl.start[A] = total;
  }
  tl.A = A;
  __syncthreads();
}

// Largest finite magnitude of N floats; infinities among them become NaN (rare:
// the second pass runs only when there are some).
template <int N>
__device__ __forceinline__ float finite_amax(float* f) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) m = fmaxf(m, fabsf(f[j]));
  if (!(m < INFINITY)) {
    m = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      f[j] = inf_to_nan(f[j]);
      m = fmaxf(m, fabsf(f[j]));
    }
  }
  return m;
}

// 32 floats times inv as 32 e4m3 bytes at a shared-memory address.
__device__ __forceinline__ void quantize32(const float* f, float inv, uint32_t dst) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* v = f + 16 * h + 4 * i;
      o[i] = cvt_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    }
    sts128(dst + 16 * h, o[0], o[1], o[2], o[3]);
  }
}

// Running largest magnitudes of the two halves of BF16 pairs (NaN is passed over).
__device__ __forceinline__ uint32_t bf16x2_absmax(uint32_t m, uint32_t p) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(p & 0x7fff7fffu));
  return r;
}
__device__ __forceinline__ float bf16x2_max(uint32_t m) {
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}
__device__ __forceinline__ uint32_t bf16x2_inf_to_nan(uint32_t p) {
  return p | ((p & 0x7fffu) == 0x7f80u ? 0x7fu : 0u) | ((p & 0x7fff0000u) == 0x7f800000u ? 0x7f0000u : 0u);
}

// Four BF16 values (two pairs, low half first) times inv as four e4m3 bytes.
__device__ __forceinline__ uint32_t quantize_bf16x4(uint32_t p0, uint32_t p1, float inv) {
  return cvt_e4m3x4(__uint_as_float(p0 << 16) * inv, __uint_as_float(p0 & 0xffff0000u) * inv,
                    __uint_as_float(p1 << 16) * inv, __uint_as_float(p1 & 0xffff0000u) * inv);
}

// Copies `bytes` (a multiple of 16) of this thread's staging slot to global
// memory; the thread wrote them itself, so only its own writes need ordering
// before the copy (fence_proxy_async_smem).
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
}
// `bytes` (a multiple of 16) from global to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// This thread's copies have read shared memory / have finished.
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// a += s * v on two FP32 values at once (each rounded as one fused multiply-add).
__device__ __forceinline__ void fma2(uint64_t& a, uint64_t s, uint32_t v0, uint32_t v1) {
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%2, %3};\n\tfma.rn.f32x2 %0, %1, v, %0;\n\t}"
      : "+l"(a)
      : "l"(s), "r"(v0), "r"(v1));
}
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
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
  const uint32_t stg_base = base + S * kStage8;
  const uint32_t bars = stg_base + 256 * kSlot8;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (S + s); };
  auto acc_full = [&](int b) { return bars + 8u * (2 * S + b); };
  auto acc_empty = [&](int b) { return bars + 8u * (2 * S + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (2 * S + 4);
  const uint32_t amax_bar = bars + 8u * (2 * S + 5);
  const uint32_t gu_bar = bars + 8u * (2 * S + 6);
  const uint32_t slot_free = bars + 8u * (2 * S + 7);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 8u * (2 * S + 8));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* row_amax = reinterpret_cast<float*>(tmem_slot + 4);                 // [2 tiles][2][128]
  int32_t* warp_tot = reinterpret_cast<int32_t*>(row_amax + 4 * kRows8);     // [32]
  TileList8 list;
  list.start = warp_tot + 32;                                                // [E + 1]
  list.seg = list.start + p.E + 1;                                           // [E + 1]
  list.id = reinterpret_cast<uint16_t*>(list.seg + p.E + 1);                 // [E]

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
    mbar_init(gu_bar, 32);
    mbar_init(slot_free, kEpiWarps8);
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

  build_tiles8(p, list, warp_tot);
  const int total = list.start[list.A];
  const int nkb = (p.R + 127) / 128;      // blocks of the reduction
  const int f_half = p.N >> 1;            // SwiGLU: first up row

  if (warp < kEpiWarp8) {
  reg_dec<kRegsCopy>();
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_a = l2_policy_evict_last();
      const uint64_t pol_w = l2_policy_evict_first();
      int st = 0;
      uint32_t ph = 0;
      long long issued = 0;
      bool ok = true;
      Tile8 tl;
      tl.a = 0;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        tl = tile8_at(list, t, tl.a);
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
  } else if (kGluBwd && warp == 3) {
    // ------------------------------------------------------------ checkpoint rows
    // For the 256 staging slots (row, half) of each tile: the row's 128 bytes
    // of g and of u by bulk copy, and its four plus four E8M0 scales.
    bool ok = true, any = false;
    int li = 0;
    Tile8 tl;
    tl.a = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x, ++li) {
      tl = tile8_at(list, t, tl.a);
      ok = mbar_wait(slot_free, static_cast<uint32_t>(li & 1), abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint32_t valid = 0;
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const int row = tl.row0 + (i & 3) * 32 + lane, f0 = tl.ft * 256 + (i >> 2) * 128;
        if (row >= tl.row_end || f0 >= p.K) continue;
        ++valid;
        const uint8_t* sc = p.saved_scales + static_cast<int64_t>(f0 / 32) * p.M + row;
        uint32_t g = 0, u = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          g |= static_cast<uint32_t>(__ldg(sc + static_cast<int64_t>(c) * p.M)) << (8 * c);
          u |= static_cast<uint32_t>(__ldg(sc + static_cast<int64_t>(c + p.K / 32) * p.M)) << (8 * c);
        }
        sts64(stg_base + static_cast<uint32_t>(i * 32 + lane) * kSlot8 + 256u, g, u);
      }
      mbar_arrive_expect_tx(gu_bar, 256 * valid);
      any = true;
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const int row = tl.row0 + (i & 3) * 32 + lane, f0 = tl.ft * 256 + (i >> 2) * 128;
        if (row >= tl.row_end || f0 >= p.K) continue;
        const uint8_t* src = p.saved + static_cast<int64_t>(row) * (2 * p.K) + f0;
        const uint32_t dst = stg_base + static_cast<uint32_t>(i * 32 + lane) * kSlot8;
        bulk_load(dst, src, 128, gu_bar);
        bulk_load(dst + 128u, src + p.K, 128, gu_bar);
      }
    }
    // an abort after some copies: they land before the CTA can exit
    if (!ok && any) mbar_drain(gu_bar, static_cast<uint32_t>((li - 1) & 1));
    __syncwarp();
  }
  } else {
    // ------------------------------------------------------------ scaled sum and epilogue
    reg_inc<kRegsEpi>();
    const int q = warp & 3;                      // tensor-memory lane quarter
    const int wg = (warp - kEpiWarp8) >> 2;      // column half
    const int r_in = q * 32 + lane;              // row of the tile
    const uint32_t tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t slot = stg_base + static_cast<uint32_t>(threadIdx.x - 32 * kEpiWarp8) * kSlot8;
    // This thread's 128 columns in two halves of 64: plain, one box; SwiGLU,
    // 64 gate columns and the 64 matching up columns.
    const uint32_t col0 = kGlu ? static_cast<uint32_t>(wg * 64) : static_cast<uint32_t>(wg * 128);
    const uint32_t col1 = kGlu ? 128u + static_cast<uint32_t>(wg * 64) : col0 + 64u;
    const int KB = (p.K + 127) / 128, NB = (p.N + 127) / 128;
    const int w_step = BWD ? KB : 1;             // weight scales of consecutive reduction blocks
    // Where a tile's scales are: the row's (stride M) and, for the two column
    // halves, the weight blocks' (stride w_step). Blocks past the last feature
    // (a tile that ends early) are clamped; their columns are not stored.
    struct Scales {
      const float *a, *w0, *w1;
    };
    auto scales_of = [&](const Tile8& tl) {
      const float* swe = p.w_scales + static_cast<int64_t>(tl.e) * NB * KB;
      const int b0 = kGlu ? tl.ft : min(tl.ft * 2 + wg, (BWD ? KB : NB) - 1);
      const int b1 = kGlu ? f_half / 128 + tl.ft : b0;
      return Scales{p.a_scales + min(tl.row0 + r_in, p.M - 1),
                    BWD ? swe + b0 : swe + static_cast<int64_t>(b0) * KB,
                    BWD ? swe + b1 : swe + static_cast<int64_t>(b1) * KB};
    };
    long long it = 0;
    int li = 0;                                  // this CTA's tile count
    Tile8 tl;
    Scales sc;
    float na = 0.0f, n0 = 0.0f, n1 = 0.0f;       // scales of the next reduction block
    if (static_cast<int>(blockIdx.x) < total) {
      tl = tile8_at(list, blockIdx.x, 0);
      sc = scales_of(tl);
      na = __ldg(sc.a);
      n0 = __ldg(sc.w0);
      if constexpr (kGlu) n1 = __ldg(sc.w1);
    }
    for (int t = blockIdx.x; t < total; t += gridDim.x, ++li) {
      const int row = tl.row0 + r_in;
      const bool row_ok = row < tl.row_end;
      const int ft = tl.ft;
      uint64_t acc2[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc2[j] = 0ull;
      bool ok = true;
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        if constexpr (kGluBwd) {
          // Once the previous tile's output has left the staging slots, warp 3
          // brings this tile's g and u there while the product runs.
          if (kb == min(2, nkb - 1)) {
            bulk_wait_read();
            __syncwarp();
            if (lane == 0) mbar_arrive(slot_free);
          }
        }
        const float s0 = na * n0, s1 = kGlu ? na * n1 : s0;
        if (kb + 1 < nkb) {
          na = __ldg(sc.a + static_cast<int64_t>(kb + 1) * p.M);
          n0 = __ldg(sc.w0 + (kb + 1) * w_step);
          if constexpr (kGlu) n1 = __ldg(sc.w1 + (kb + 1) * w_step);
        } else if (t + static_cast<int>(gridDim.x) < total) {
          // the next tile's first scales arrive during this tile's epilogue
          tl = tile8_at(list, t + gridDim.x, tl.a);
          sc = scales_of(tl);
          na = __ldg(sc.a);
          n0 = __ldg(sc.w0);
          if constexpr (kGlu) n1 = __ldg(sc.w1);
        }
        const int b = static_cast<int>(it & 1);
        const bool r = mbar_wait(acc_full(b), static_cast<uint32_t>((it >> 1) & 1), abort_flag);
        if (!__shfl_sync(0xffffffffu, r ? 1 : 0, 0)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tb = tq + static_cast<uint32_t>(b) * 256u;
        // Four chunks of 32 columns, the next one loaded while this one is added.
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(tb + col0, v[0]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c < 3) tmem_ld_32x32b_x32(tb + (c < 1 ? col0 + 32u : col1 + 32u * (c - 1)), v[(c + 1) & 1]);
          const float s = c < 2 ? s0 : s1;
          const uint64_t ss = pair2(s, s);
#pragma unroll
          for (int j = 0; j < 16; ++j) fma2(acc2[16 * c + j], ss, v[c & 1][2 * j], v[c & 1][2 * j + 1]);
          if (c < 3) tmem_wait_ld();
          if (c == 2) {               // everything is in registers: the buffer is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty(b));
          }
        }
      }
      if constexpr (kGluBwd) {
        if (ok) ok = mbar_wait(gu_bar, static_cast<uint32_t>(li & 1), abort_flag);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) break;
      [[maybe_unused]] float acc[128];
      if constexpr (!kGluBwd) {
#pragma unroll
        for (int j = 0; j < 64; ++j) unpair2(acc2[j], acc[2 * j], acc[2 * j + 1]);
      }
      if constexpr (!kGluBwd) bulk_wait_read();  // the previous tile's output has left the slot

      if constexpr (kGlu) {
        // acc[0..63] gate, acc[64..127] up of features f0 ..; the slot holds
        // [64 B h][64 B gate][64 B up].
        const int f0 = ft * 128 + wg * 64;
        if (p.saved != nullptr) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int e = fp8_block_exp(finite_amax<32>(acc + 32 * c));
            quantize32(acc + 32 * c, exp2_int(-e), slot + 64u + 32u * c);
            const int grp = ((c < 2 ? f0 : f_half + f0) >> 5) + (c & 1);
            if (row_ok) p.saved_scales[static_cast<int64_t>(grp) * p.M + row] = static_cast<uint8_t>(e + 127);
          }
        }
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[j] = silu_f(acc[j]) * acc[64 + j];
        float m = finite_amax<64>(acc);
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
        const int e = fp8_block_exp(m);
        quantize32(acc, exp2_int(-e), slot);
        quantize32(acc + 32, exp2_int(-e), slot + 32u);
        fence_proxy_async_smem();
        if (row_ok) {
          bulk_store(p.out + static_cast<int64_t>(row) * f_half + f0, slot, 64);
          if (p.saved != nullptr) {
            uint8_t* sv = p.saved + static_cast<int64_t>(row) * p.N + f0;
            bulk_store(sv, slot + 64u, 64);
            bulk_store(sv + f_half, slot + 128u, 64);
          }
          if (wg == 0) p.out_scales[static_cast<int64_t>(ft) * p.M + row] = exp2_int(e);
        }
      } else if constexpr (kGluBwd) {
        // dh of features f0 .. f0 + 127; the slot holds [128 B g][128 B u][4 + 4
        // scales] and then [128 B dg][128 B du].
        const int f0 = ft * 256 + wg * 128;
        const int K = p.K;
        {
          const uint2 gu_scales = lds64(slot + 256u);
          uint32_t mg = 0u, mu = 0u;            // largest magnitudes of even and odd features, BF16 pairs
          // Each pair of dh is replaced by the BF16 pairs dg and du of its two features.
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float sg = e8m0_to_float((gu_scales.x >> (8 * c)) & 0xffu);
            const float su = e8m0_to_float((gu_scales.y >> (8 * c)) & 0xffu);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 g4 = lds128(slot + 32u * c + 16u * h);
              const uint4 u4 = lds128(slot + 128u + 32u * c + 16u * h);
              const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 g2 = e4m3x2_to_float2(gw[i >> 1] >> (16 * (i & 1)));
                const float2 u2 = e4m3x2_to_float2(uw[i >> 1] >> (16 * (i & 1)));
                const int a = 16 * c + 8 * h + i;
                float dh[2], dg[2], du[2];
                unpair2(acc2[a], dh[0], dh[1]);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const float g = (z ? g2.y : g2.x) * sg, u = (z ? u2.y : u2.x) * su;
                  const float s = sigmoid_f(g), x = dh[z];
                  dg[z] = x * u * s * (1.0f + g * (1.0f - s));
                  du[z] = x * g * s;
                }
                const uint32_t pg = pack_bf16x2(dg[0], dg[1]), pu = pack_bf16x2(du[0], du[1]);
                mg = bf16x2_absmax(mg, pg);
                mu = bf16x2_absmax(mu, pu);
                acc2[a] = pair2(__uint_as_float(pg), __uint_as_float(pu));
              }
            }
          }
          float ag = bf16x2_max(mg), au = bf16x2_max(mu);
          if (!(ag < INFINITY) || !(au < INFINITY)) {   // infinities become NaN (rare)
            mg = mu = 0u;
#pragma unroll
            for (int j = 0; j < 64; ++j) {
              float pg, pu;
              unpair2(acc2[j], pg, pu);
              const uint32_t wg_ = bf16x2_inf_to_nan(__float_as_uint(pg));
              const uint32_t wu_ = bf16x2_inf_to_nan(__float_as_uint(pu));
              mg = bf16x2_absmax(mg, wg_);
              mu = bf16x2_absmax(mu, wu_);
              acc2[j] = pair2(__uint_as_float(wg_), __uint_as_float(wu_));
            }
            ag = bf16x2_max(mg);
            au = bf16x2_max(mu);
          }
          const int eg = fp8_block_exp(ag), eu = fp8_block_exp(au);
          const float ig = exp2_int(-eg), iu = exp2_int(-eu);
          // 16 features at a time: eight pairs give 16 bytes of dg and of du.
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t og[4], ou[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float g0, u0, g1, u1;
              unpair2(acc2[8 * c + 2 * i], g0, u0);
              unpair2(acc2[8 * c + 2 * i + 1], g1, u1);
              og[i] = quantize_bf16x4(__float_as_uint(g0), __float_as_uint(g1), ig);
              ou[i] = quantize_bf16x4(__float_as_uint(u0), __float_as_uint(u1), iu);
            }
            sts128(slot + 16u * c, og[0], og[1], og[2], og[3]);
            sts128(slot + 128u + 16u * c, ou[0], ou[1], ou[2], ou[3]);
          }
          fence_proxy_async_smem();
          if (row_ok && f0 < K) {
          uint8_t* dst = p.out + static_cast<int64_t>(row) * (2 * K) + f0;
          bulk_store(dst, slot, 128);
          bulk_store(dst + K, slot + 128u, 128);
          const int64_t blk = f0 / 128;
          p.out_scales[blk * p.M + row] = exp2_int(eg);
          p.out_scales[(blk + K / 128) * p.M + row] = exp2_int(eu);
          }
        }
      } else {
        const int F = BWD ? p.K : p.N;
        const int f0 = ft * 256 + wg * 128;
#pragma unroll
        for (int c = 0; c < 16; ++c)
          sts128(slot + 16u * c, pack_bf16x2(acc[8 * c], acc[8 * c + 1]),
                 pack_bf16x2(acc[8 * c + 2], acc[8 * c + 3]), pack_bf16x2(acc[8 * c + 4], acc[8 * c + 5]),
                 pack_bf16x2(acc[8 * c + 6], acc[8 * c + 7]));
        fence_proxy_async_smem();
        if (row_ok && f0 < F)          // F % 16 == 0: whole 32-byte pieces
          bulk_store(p.out + 2 * (static_cast<int64_t>(row) * F + f0), slot,
                     2u * static_cast<uint32_t>(min(128, F - f0)));
      }
      bulk_commit();
    }
    bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, 512);
}

}  // namespace

cudaError_t launch_grouped_fp8_gemm(bool bwd, int epi, const CUtensorMap& ta, const CUtensorMap& tw,
                                    const Fp8GemmArgs& p, int grid, cudaStream_t s) {
  const size_t smem = smem_bytes8(p.E);
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
