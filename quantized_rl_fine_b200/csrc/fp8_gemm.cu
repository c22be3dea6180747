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
// lie inside one thread, which the quantizing epilogues use. The sum of scaled
// blocks cannot stay in the tensor core: weight scales are any FP32 numbers.
//
// Experts of many rows: CTA pairs share a tile of 256 rows (cta_group::2, each
// CTA brings its own rows and half the weights). Experts of few rows: tiles of
// 32 or 64 rows, whose stages hold little but weights, so that more are in
// flight. All forms add the same numbers in the same order and give the same bits.
//
// What bounds it. Few rows: the weight stream (a block of 256 x 128 weights is
// 32 KiB, 0.73 us at 6.56 TB/s over 148 SMs; the four MMAs take 0.3). Measured: 16
// tokens of 8 of 48 experts, K 7168, N 4096 with SwiGLU 205 us (1.41 GB,
// 6.9 TB/s with what L2 keeps between calls); one token of 8 experts 43 us (5.4 TB/s: one tile a CTA, filling and
// draining its pipeline counts); 62 rows x 64 experts of 2048 x 2048 57 us (5.3 TB/s).
// Many rows: the hand-over between tensor core and epilogue. Per 128 x 256 x 128
// block the MMAs alone take 565 cycles, with barriers but no tensor-memory
// reads 768, complete about 970: commit, wake-up, two rounds of
// tensor-memory loads and the release follow one another, and only two buffers
// of 256 columns fit. 768 rows x 48 experts, K 7168, N 4096: 1037 us at full
// clocks (2.09 PFLOP/s), 1190 under the power cap; backward 1074 / 1248; SwiGLU
// 1040 / 1225, with checkpoint 1078 / 1275 (its epilogue, about 2 us a tile, is
// not overlapped: the accumulators are in registers). SwiGLU backward 607 us for
// half the work.
// Tried, without gain: two MMA issuers, spinning waits, tensor-memory loads held
// over the loop's back edge (the compiler cannot keep the registers). 128-column
// tiles and a column split with their own barriers gained nothing while the
// epilogue threads loaded the scales themselves, which then bounded a block
// whatever its width; they have not been measured since the scale warp does.
//
// The backward reads the same weights in place, as the MN-major B operand:
// features contiguous, 128-byte swizzled blocks of 128 features.
//
// Every wait is bounded; on a timeout the kernel records a device error, all
// roles stop (in a pair, both CTAs'), the copies and MMAs in flight finish (again
// bounded), tensor memory is freed and the kernel returns.
#include <algorithm>
#include <atomic>

#include "fp8.cuh"
#include "fp8_gemm.cuh"
#include "fp8_wait.cuh"

namespace moeq {

namespace {

constexpr int kRows8 = 128;              // token rows per tile (MMA M)
constexpr uint32_t kBoxBytes = 16384;    // one operand box: 128 rows x 128 bytes
// Four forms: single CTAs on 128 token rows, pairs on 256, and single CTAs on
// 32 or 64 rows for experts of few rows.
constexpr int kSingle8 = 0, kPair8 = 1, kFew8 = 2, kSome8 = 3;
// Lane quarters with rows in one CTA, hence epilogue warps and staging slots in use.
__host__ __device__ constexpr int quarters8(int form) { return form == kFew8 ? 1 : form == kSome8 ? 2 : 4; }
__host__ __device__ constexpr int tile_rows8(int form) { return form == kPair8 ? 256 : 32 * quarters8(form); }
// One stage: the CTA's token rows and two weight boxes (one in a pair). The MMA
// always reads 128 rows of A; with fewer loaded the others are the weight
// boxes behind them, and their products are not looked at.
__host__ __device__ constexpr uint32_t row_bytes8(int form) { return 4096u * quarters8(form); }
__host__ __device__ constexpr uint32_t stage_bytes8(int form) {
  return row_bytes8(form) + (form == kPair8 ? 1u : 2u) * kBoxBytes;
}
__host__ __device__ constexpr int stages8(int form) { return form == kSingle8 ? 3 : form == kFew8 ? 5 : 4; }
constexpr int kEpiWarp8 = 4;             // warp 0 copies, warp 1 issues MMAs, warps 4-11 epilogue
constexpr int kEpiWarps8 = 8;
constexpr int kThreads8 = 32 * (kEpiWarp8 + kEpiWarps8);
// Registers: 168 a thread at launch (384 x 168 = 64512); the first warpgroup
// gives up 96 a thread and the two epilogue warpgroups take 48 each: 128 x 72
// + 256 x 216 = 64512. An epilogue thread holds 128 accumulators and 64 values in flight.
constexpr int kRegsCopy = 72, kRegsEpi = 216;
static_assert(128 * kRegsCopy + 256 * kRegsEpi <= kThreads8 * 168, "register split");
// Output staging of one epilogue thread: its 256 bytes of a row, padded so
// that the 16-byte stores of eight neighbouring threads fall in distinct banks.
constexpr uint32_t kSlot8 = 272;
__host__ __device__ constexpr uint32_t slots_bytes8(int form) { return 64u * quarters8(form) * kSlot8; }
constexpr size_t smem_bytes8(int E, int form) {
  return 1024 + stages8(form) * stage_bytes8(form) + slots_bytes8(form) + 8 * (2 * stages8(form) + 10) + 16 + 4 * 4 * kRows8 + 4 * 32 +
         4 * 2 * (static_cast<size_t>(E) + 1) + 2 * static_cast<size_t>(E);
}
static_assert(smem_bytes8(1024, 0) <= 227 * 1024 && smem_bytes8(1024, 1) <= 227 * 1024 &&
                  smem_bytes8(1024, 2) <= 227 * 1024 && smem_bytes8(1024, 3) <= 227 * 1024, "shared memory of the largest stack");

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

// The same over a pair: D and A 128 rows in each CTA, B's N rows split between
// them (even CTA [0, N/2)), M = 256.
__device__ __forceinline__ void mma_f8_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, {%5, %5, %5, %5, %5, %5, %5, %5}, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(0u)
      : "memory");
}

// Box of 128-byte rows; in a pair `bar` may be the other CTA's barrier (a
// cluster address). No multicast: each CTA brings its own boxes.
template <int PAIR>
__device__ __forceinline__ void tma_load8(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0,
                                          int32_t c1, int32_t c2, uint64_t policy) {
  if constexpr (PAIR) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
        : "memory");
  } else {
    tma_load_3d_hint(dst, map, bar, c0, c1, c2, policy);
  }
}

// Arrival on the other CTA's barrier with the default (CTA) release: what it
// hands over is tensor memory, ordered by the tcgen05 fence before it. A
// cluster-scope release here, or a cluster-scope acquire in the wait, cost
// 1.5 us per reduction block (the product 2.2x slower).
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// mbar_wait with few registers held: time in 32 bits, the abort flag by its
// shared-memory address, the budget (2^41 cycles at most) read when asked. In
// a pair both CTAs' flags are set, so that the other one soon stops too.
template <int PAIR>
__device__ __forceinline__ bool mbar_wait8(uint32_t bar, uint32_t parity, uint32_t abort_flag) {
  if (mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) return true;
  const uint32_t t0 = wait_units(clock64());
  while (!mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) {
    uint32_t gone;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(gone) : "r"(abort_flag));
    if (gone) return false;
    if (wait_spent(t0, wait_units(clock64()), *reinterpret_cast<volatile long long*>(&g_wait_budget))) {
      raise_device_error(MOE_DEVERR_WAIT_TIMEOUT);
      if constexpr (PAIR) {
        for (uint32_t r = 0; r < 2; ++r)
          asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(abort_flag, r)), "r"(1u)
                       : "memory");
      } else {
        asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort_flag), "r"(1u));
      }
      return false;
    }
  }
  return true;
}

// The full barriers of a CTA's stages, for close_fills.
struct FullBars8 {
  uint32_t first, stage_bytes;
  __device__ __forceinline__ void add_bytes(uint32_t s) const {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(first + 8u * s), "r"(stage_bytes)
                 : "memory");
  }
  __device__ __forceinline__ void arrive(uint32_t s) const { mbar_arrive_expect_tx(first + 8u * s, stage_bytes); }
  __device__ __forceinline__ void wait(uint32_t s, uint32_t parity) const { mbar_drain(first + 8u * s, parity); }
};

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
template <int FORM>
__device__ __forceinline__ Tile8 tile8_at(const TileList8& tl, int t, int a0, int rank) {
  constexpr int kTileRows = tile_rows8(FORM);
  int lo = a0, hi = tl.A - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tl.start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  Tile8 r;
  r.a = lo;
  r.e = tl.id[lo];
  const int seg0 = tl.seg[lo], seg1 = tl.seg[lo + 1];
  const int nrt = (seg1 - seg0 + kTileRows - 1) / kTileRows;
  const int local = t - tl.start[lo];
  r.ft = local / nrt;
  r.row0 = seg0 + (local - r.ft * nrt) * kTileRows + rank * kRows8;
  r.row_end = min(seg1, r.row0 + min(kTileRows, kRows8));
  return r;
}

// Builds the list; the active experts' rows must lie behind one another from
// 0 to M. Tables that do not say so (or name an expert outside the stack) give
// an empty list and the device error.
template <int FORM>
__device__ void build_tiles8(const Fp8GemmArgs& p, TileList8& tl, int32_t* warp_tot) {
  constexpr int kTileRows = tile_rows8(FORM);
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
    local += p.n_ftiles * ((s1 - s0 + kTileRows - 1) / kTileRows);
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
    run += p.n_ftiles * ((tl.seg[a + 1] - tl.seg[a] + kTileRows - 1) / kTileRows);
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

// `bytes` (a multiple of 16) from global to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Stores BYTES of each of the warp's 32 staging slots, rows [0, valid), to rows
// of ld bytes at dst: BYTES / 16 neighbouring lanes a row, so that a store
// instruction writes whole sectors of several rows. (Bulk copies of a row's 64
// bytes, one a lane, took 2 us a tile more: 1536 rows x 48 experts, K 2048, N 7168,
// SwiGLU with checkpoint 1485 us instead of 1280.)
template <int BYTES>
__device__ __forceinline__ void store_rows(uint8_t* dst, int64_t ld, uint32_t slot0, int valid, int lane,
                                           uint32_t bytes = BYTES) {
  constexpr int L = BYTES / 16, kRowsAtOnce = 32 / L;
  const int r0 = lane / L;
  const uint32_t c = 16u * (lane % L);
  uint32_t src = slot0 + static_cast<uint32_t>(r0) * kSlot8 + c;
  uint8_t* d = dst + r0 * ld + c;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    if (r0 + i * kRowsAtOnce < valid && c < bytes) *reinterpret_cast<uint4*>(d) = lds128(src);
    src += kRowsAtOnce * kSlot8;
    d += kRowsAtOnce * ld;
  }
}

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
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t a) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(a) : "memory");
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

template <int BWD, int EPI, int FORM>
__global__ void __launch_bounds__(kThreads8, 1)
grouped_fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm_a,
                        const __grid_constant__ CUtensorMap tm_w, const Fp8GemmArgs p) {
  constexpr int PAIR = FORM == kPair8 ? 1 : 0;
  constexpr int kQuarters = quarters8(FORM);
  constexpr int kActive = 2 * kQuarters;         // epilogue warps with rows
  constexpr bool kGlu = !BWD && EPI == MOE_EPI_SWIGLU;
  constexpr bool kGluBwd = BWD && EPI == MOE_EPI_SWIGLU_BWD;
  extern __shared__ uint8_t smem_raw8[];
  const uint32_t raw = smem_u32(smem_raw8);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw8 + (base - raw);
  constexpr int S = stages8(FORM);
  constexpr uint32_t kStage8 = stage_bytes8(FORM);
  auto A_at = [&](int s) { return base + s * kStage8; };
  auto B_at = [&](int s) { return base + s * kStage8 + row_bytes8(FORM); };
  const uint32_t stg_base = base + S * kStage8;
  const uint32_t bars = stg_base + slots_bytes8(FORM);
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (S + s); };
  auto acc_full = [&](int b) { return bars + 8u * (2 * S + b); };      // accumulator buffer b (two)
  auto acc_empty = [&](int b) { return bars + 8u * (2 * S + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (2 * S + 4);
  const uint32_t amax_bar = bars + 8u * (2 * S + 5);
  const uint32_t gu_bar = bars + 8u * (2 * S + 6);
  const uint32_t slot_free = bars + 8u * (2 * S + 7);
  auto sc_free = [&](int b) { return bars + 8u * (2 * S + 8 + b); };   // scales of buffer b have been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 8u * (2 * S + 10));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t abort_at = bars + 8u * (2 * S + 10) + 4u;
  // What the copying warps have begun: stage fills, and tiles' checkpoint rows.
  const uint32_t fills_at = abort_at + 4u, ck_tiles_at = abort_at + 8u;
  float* row_amax = reinterpret_cast<float*>(tmem_slot + 4);                 // [2 tiles][2][128]
  int32_t* warp_tot = reinterpret_cast<int32_t*>(row_amax + 4 * kRows8);     // [32]
  TileList8 list;
  list.start = warp_tot + 32;                                                // [E + 1]
  list.seg = list.start + p.E + 1;                                           // [E + 1]
  list.id = reinterpret_cast<uint16_t*>(list.seg + p.E + 1);                 // [E]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Position in the pair (0 issues the MMAs) and the tile walk.
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int t_first = static_cast<int>(blockIdx.x) >> PAIR;
  const int t_step = static_cast<int>(gridDim.x) >> PAIR;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 2);               // the MMAs' commit and the scale warp
      mbar_init(acc_empty(b), kActive << PAIR);
      mbar_init(sc_free(b), kActive);
    }
    mbar_init(drain_bar, 1);
    mbar_init(amax_bar, kActive);
    mbar_init(gu_bar, 32);
    mbar_init(slot_free, kActive);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_w);
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_alloc_pair(smem_u32(tmem_slot), 512);
    else tmem_alloc(smem_u32(tmem_slot), 512);
  }
  tc_fence_before();
  // (a pair also waits until the other CTA's barriers are initialised)
  if constexpr (PAIR) cluster_sync_all(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();

  build_tiles8<FORM>(p, list, warp_tot);
  const int total = list.start[list.A];
  const int nkb = p.nkb;                  // blocks of the reduction
  const int f_half = p.N >> 1;            // SwiGLU: first up row

  if (warp < kEpiWarp8) reg_dec<kRegsCopy>();
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_a = l2_policy_evict_last();
      const uint64_t pol_w = p.w_once ? l2_policy_evict_first() : l2_policy_evict_last();
      int st = 0;
      uint32_t ph = 0, fills = 0;
      bool ok = true;
      Tile8 tl;
      tl.a = 0;
      for (int t = t_first; t < total && ok; t += t_step) {
        tl = tile8_at<FORM>(list, t, tl.a, rank);
        const int c0 = kGlu ? tl.ft * 128 : tl.ft * 256;       // features of the two boxes
        const int c1 = kGlu ? f_half + tl.ft * 128 : c0 + 128;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait8<PAIR>(empty(st), ph ^ 1u, abort_at)) { ok = false; break; }
          // A pair's stages are one: both CTAs' copies count on the even CTA's
          // barrier, which is where the MMAs are issued.
          uint32_t bar = full(st);
          if constexpr (PAIR) bar = cluster_addr(bar, 0);
          if (rank == 0) mbar_arrive_expect_tx(full(st), kStage8 << PAIR);
          tma_load8<PAIR>(A_at(st), &tm_a, bar, kb * 128, tl.row0, 0, pol_a);
          // weight boxes: both, or in a pair the CTA's own half of the features
          const int cf = rank == 1 ? c1 : c0;
          if constexpr (BWD) {
            tma_load8<PAIR>(B_at(st), &tm_w, bar, cf, kb * 128, tl.e, pol_w);
            if constexpr (!PAIR) tma_load8<PAIR>(B_at(st) + kBoxBytes, &tm_w, bar, c1, kb * 128, tl.e, pol_w);
          } else {
            tma_load8<PAIR>(B_at(st), &tm_w, bar, kb * 128, cf, tl.e, pol_w);
            if constexpr (!PAIR) tma_load8<PAIR>(B_at(st) + kBoxBytes, &tm_w, bar, kb * 128, c1, tl.e, pol_w);
          }
          ++fills;
          if (++st == S) { st = 0; ph ^= 1u; }
        }
      }
      sts32(fills_at, fills);
      if constexpr (PAIR) {
        // The even CTA's commits arrive here too, after the last stages as well:
        // the CTA stays until they have.
        for (int i = 0; i < S && ok && rank == 1; ++i) {
          ok = mbar_wait8<PAIR>(empty(st), ph ^ 1u, abort_at);
          if (++st == S) { st = 0; ph ^= 1u; }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc = idesc_f8(kRows8 << PAIR, 256, BWD ? 1u : 0u);
    int st = 0;
    uint32_t ph = 0;
    uint32_t it = 0;                      // reduction blocks handed over (buffer it % 2)
    bool ok = true;
    auto wait_w = [&](uint32_t bar, uint32_t parity) {
      const bool r = mbar_wait8<PAIR>(bar, parity, abort_at);
      return __shfl_sync(0xffffffffu, r ? 1 : 0, 0) != 0;
    };
    auto commit = [](uint32_t bar) {
      if constexpr (PAIR) mma_commit_pair(bar, 3); else mma_commit(bar);
    };
    for (int t = t_first; t < total && ok; t += t_step) {
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const int b = static_cast<int>(it & 1);
        if (!wait_w(full(st), ph)) { ok = false; break; }
        if (!wait_w(acc_empty(b), static_cast<uint32_t>((it >> 1) & 1) ^ 1u)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d = tmem_base + static_cast<uint32_t>(b) * 256u;
          const uint64_t da = smem_desc_sw128(A_at(st), 16, 1024);
          const uint64_t db = BWD ? smem_desc_sw128(B_at(st), kBoxBytes, 1024)
                                  : smem_desc_sw128(B_at(st), 16, 1024);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {  // 32 of the 128 reduction elements each
            const uint64_t bk = db + (BWD ? 256 : 2) * ks;
            if constexpr (PAIR) mma_f8_ss_pair(d, da + 2 * ks, bk, idesc, ks > 0 ? 1u : 0u);
            else mma_f8_ss(d, da + 2 * ks, bk, idesc, ks > 0 ? 1u : 0u);
          }
          commit(empty(st));
          commit(acc_full(b));
        }
        __syncwarp();
        if (++st == S) { st = 0; ph ^= 1u; }
      }
    }
    if (elect_one()) commit(drain_bar);
    __syncwarp();
    if (lane == 0) mbar_drain(drain_bar, 0);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ scales
    // Forms each reduction block's factors (row scale times weight scale) two
    // blocks ahead and hands them over with the accumulator buffer, in the
    // padding of the epilogue threads' slots. Loaded by the epilogue threads
    // themselves one block ahead, they bounded the product: a block took as
    // long as such a load, about 1000 cycles, however few columns it had.
    bool ok = true;
    uint32_t it = 0;
    Tile8 tl;
    tl.a = 0;
    for (int t = t_first; t < total && ok; t += t_step) {
      tl = tile8_at<FORM>(list, t, tl.a, rank);
      // Blocks past the last feature (a tile that ends early) are clamped;
      // their columns are not stored.
      const float* pw = p.w_scales + static_cast<int64_t>(tl.e) * p.NB * p.KB;
      int64_t up = 0;                        // from the first to the second half's weight block
      if constexpr (BWD) {
        pw += tl.ft * 2;
        up = min(tl.ft * 2 + 1, p.KB - 1) - tl.ft * 2;
      } else if constexpr (kGlu) {
        pw += static_cast<int64_t>(tl.ft) * p.KB;
        up = static_cast<int64_t>(f_half / 128) * p.KB;
      } else {
        pw += static_cast<int64_t>(tl.ft * 2) * p.KB;
        up = static_cast<int64_t>(min(tl.ft * 2 + 1, p.NB - 1) - tl.ft * 2) * p.KB;
      }
      const float* pa = p.a_scales;
      int off[kQuarters];
#pragma unroll
      for (int i = 0; i < kQuarters; ++i) off[i] = min(tl.row0 + 32 * i + lane, p.M - 1);
      struct Set {
        float a[kQuarters], w0, w1;
      } set[2];
      auto fetch = [&](Set& x) {
#pragma unroll
        for (int i = 0; i < kQuarters; ++i) x.a[i] = __ldg(pa + off[i]);
        x.w0 = __ldg(pw);
        x.w1 = __ldg(pw + up);
        pa += p.M;
        pw += BWD ? p.KB : 1;
      };
      auto step = [&](Set& x, int kb) {
        const int b = static_cast<int>(it & 1);
        ok = mbar_wait8<PAIR>(sc_free(b), ((it >> 1) & 1) ^ 1u, abort_at);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
#pragma unroll
        for (int i = 0; i < kActive; ++i) {
          const uint32_t pad = stg_base + static_cast<uint32_t>(i * 32 + lane) * kSlot8 + 256u;
          const float sa = x.a[i % kQuarters];
          if constexpr (kGlu)
            sts64(pad + 8u * b, __float_as_uint(sa * x.w0), __float_as_uint(sa * x.w1));
          else
            sts32(pad + (kGluBwd ? 8u : 0u) + 4u * b, __float_as_uint(sa * (i < kQuarters ? x.w0 : x.w1)));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_full(b));
        if (kb + 2 < p.nkb) fetch(x);
        ++it;
      };
      fetch(set[0]);
      if (p.nkb > 1) fetch(set[1]);
      for (int kb = 0; kb < p.nkb && ok; kb += 2) {
        step(set[0], kb);
        if (ok && kb + 1 < p.nkb) step(set[1], kb + 1);
      }
    }
  } else if (kGluBwd && warp == 3) {
    // ------------------------------------------------------------ checkpoint rows
    // For the staging slots (half, row) of each tile: the row's 128 bytes
    // of g and of u by bulk copy, and its four plus four E8M0 scales.
    uint32_t li = 0;
    Tile8 tl;
    tl.a = 0;
    for (int t = t_first; t < total; t += t_step, ++li) {
      tl = tile8_at<FORM>(list, t, tl.a, rank);
      const bool ok = mbar_wait8<PAIR>(slot_free, li & 1u, abort_at);
      if (!__all_sync(0xffffffffu, ok)) break;
      uint32_t valid = 0;
#pragma unroll 1
      for (int i = 0; i < kActive; ++i) {
        const int row = tl.row0 + (i % kQuarters) * 32 + lane, f0 = tl.ft * 256 + (i / kQuarters) * 128;
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
#pragma unroll 1
      for (int i = 0; i < kActive; ++i) {
        const int row = tl.row0 + (i % kQuarters) * 32 + lane, f0 = tl.ft * 256 + (i / kQuarters) * 128;
        if (row >= tl.row_end || f0 >= p.K) continue;
        const uint8_t* src = p.saved + static_cast<int64_t>(row) * (2 * p.K) + f0;
        const uint32_t dst = stg_base + static_cast<uint32_t>(i * 32 + lane) * kSlot8;
        bulk_load(dst, src, 128, gu_bar);
        bulk_load(dst + 128u, src + p.K, 128, gu_bar);
      }
    }
    if (lane == 0) sts32(ck_tiles_at, li);
    __syncwarp();
  } else if (warp >= kEpiWarp8) {
    // ------------------------------------------------------------ scaled sum and epilogue
    reg_inc<kRegsEpi>();
    const int q = warp & 3;                      // tensor-memory lane quarter
    const int wg = (warp - kEpiWarp8) >> 2;      // column half
    const int r_in = q * 32 + lane;              // row of the tile
    const uint32_t tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t slot = stg_base + static_cast<uint32_t>(wg * 32 * kQuarters + r_in) * kSlot8;
    // This thread's 128 columns in two halves of 64: plain, one box; SwiGLU,
    // 64 gate columns and the 64 matching up columns.
    const uint32_t col0 = static_cast<uint32_t>(kGlu ? wg * 64 : wg * 128);
    const uint32_t col1 = col0 + (kGlu ? 128u : 64u);
    // Registers are what this loop is short of (128 accumulators, 64 values in
    // flight, 216 a thread), and a spill in it costs more than anything else
    // here: the tile is kept as (row or -1, ft, a).
    int row = -1, ft = 0, ta = 0;
    auto enter = [&](int t) {
      const Tile8 tl = tile8_at<FORM>(list, t, ta, rank);
      ta = tl.a;
      ft = tl.ft;
      row = tl.row0 + r_in;
      if (row >= tl.row_end) row = -1;
    };
    uint32_t it = 0;                             // reduction blocks so far (buffer it % 2)
    uint32_t li = 0;                             // parity of this CTA's tile count
    // (a warp whose lane quarter has no rows has nothing to do)
    const int t_end = q < kQuarters ? total : 0;
    if (t_first < t_end) enter(t_first);
    for (int t = t_first; t < t_end; t += t_step, li ^= 1u) {
      const int cur_row = row, cur_ft = ft;
      uint64_t acc2[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc2[j] = 0ull;
      bool ok = true;
      for (int kb = 0; kb < p.nkb; ++kb, ++it) {
        if constexpr (kGluBwd) {
          // Once the previous tile's output has left the staging slots, warp 3
          // brings this tile's g and u there while the product runs.
          if (kb == min(2, p.nkb - 1) && lane == 0) mbar_arrive(slot_free);
        }
        const int b = static_cast<int>(it & 1);
        const bool r = mbar_wait8<PAIR>(acc_full(b), static_cast<uint32_t>((it >> 1) & 1), abort_at);
        if (!__shfl_sync(0xffffffffu, r ? 1 : 0, 0)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tb = tq + static_cast<uint32_t>(b) * 256u;
        // Two chunks of 32 columns in flight; the next one is requested as soon as
        // a chunk's registers are free.
        uint32_t v0[32], v1[32];
        tmem_ld_32x32b_x32(tb + col0, v0);
        tmem_ld_32x32b_x32(tb + col0 + 32u, v1);
        float s0, s1;
        if constexpr (kGlu) {
          const uint2 sc = lds64(slot + 256u + 8u * b);
          s0 = __uint_as_float(sc.x);
          s1 = __uint_as_float(sc.y);
        } else {
          s0 = s1 = __uint_as_float(lds32(slot + 256u + (kGluBwd ? 8u : 0u) + 4u * b));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tmem_wait_ld();
          if (h == 1) {                 // everything is in registers: the buffer is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (PAIR) arrive_remote(cluster_addr(acc_empty(b), 0));
              else mbar_arrive(acc_empty(b));
              mbar_arrive(sc_free(b));
            }
          }
          const float s = h ? s1 : s0;
          const uint64_t ss = pair2(s, s);
#pragma unroll
          for (int j = 0; j < 16; ++j) fma2(acc2[32 * h + j], ss, v0[2 * j], v0[2 * j + 1]);
          if (h == 0) tmem_ld_32x32b_x32(tb + col1, v0);
#pragma unroll
          for (int j = 0; j < 16; ++j) fma2(acc2[32 * h + 16 + j], ss, v1[2 * j], v1[2 * j + 1]);
          if (h == 0) tmem_ld_32x32b_x32(tb + col1 + 32u, v1);
        }
      }
      if constexpr (kGluBwd) {
        if (ok) ok = mbar_wait8<PAIR>(gu_bar, li, abort_at);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) break;
      if (t + t_step < total) enter(t + t_step);
      [[maybe_unused]] float acc[128];
      if constexpr (!kGluBwd) {
#pragma unroll
        for (int j = 0; j < 64; ++j) unpair2(acc2[j], acc[2 * j], acc[2 * j + 1]);
      }
      // The warp's rows are the first `valid` lanes, from row `first`. (Asked for
      // behind the arithmetic, which needs the registers.)
      const uint32_t slot0 = slot - static_cast<uint32_t>(lane) * kSlot8;
      int valid = 0;
      int64_t first = 0;
      auto warp_rows = [&] {
        __syncwarp();                        // the slots have been written
        valid = __popc(__ballot_sync(0xffffffffu, cur_row >= 0));
        first = __shfl_sync(0xffffffffu, cur_row, 0);
      };

      if constexpr (kGlu) {
        // acc[0..63] gate, acc[64..127] up of features f0 ..; the slot holds
        // [64 B h][64 B gate][64 B up].
        const int f0 = cur_ft * 128 + wg * 64;
        if (p.saved != nullptr) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int e = fp8_block_exp(finite_amax<32>(acc + 32 * c));
            quantize32(acc + 32 * c, exp2_int(-e), slot + 64u + 32u * c);
            const int grp = ((c < 2 ? f0 : f_half + f0) >> 5) + (c & 1);
            if (cur_row >= 0) p.saved_scales[static_cast<int64_t>(grp) * p.M + cur_row] = static_cast<uint8_t>(e + 127);
          }
        }
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[j] = silu_f(acc[j]) * acc[64 + j];
        float m = finite_amax<64>(acc);
        // The block of 128 features spans both column halves. Two exchange
        // buffers in turn: passing tile n + 1's barrier means that everybody
        // has read tile n's, which tile n + 2 then writes.
        float* xch = row_amax + li * 2 * kRows8;
        xch[wg * kRows8 + r_in] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(amax_bar);
        const bool met = mbar_wait8<PAIR>(amax_bar, li, abort_at);
        if (!__shfl_sync(0xffffffffu, met ? 1 : 0, 0)) break;
        m = fmaxf(m, xch[(wg ^ 1) * kRows8 + r_in]);
        const int e = fp8_block_exp(m);
        quantize32(acc, exp2_int(-e), slot);
        quantize32(acc + 32, exp2_int(-e), slot + 32u);
        warp_rows();
        store_rows<64>(p.out + first * f_half + f0, f_half, slot0, valid, lane);
        if (p.saved != nullptr) {
          uint8_t* sv = p.saved + first * p.N + f0;
          store_rows<64>(sv, p.N, slot0 + 64u, valid, lane);
          store_rows<64>(sv + f_half, p.N, slot0 + 128u, valid, lane);
        }
        if (wg == 0 && cur_row >= 0) p.out_scales[static_cast<int64_t>(cur_ft) * p.M + cur_row] = exp2_int(e);
      } else if constexpr (kGluBwd) {
        // dh of features f0 .. f0 + 127; the slot holds [128 B g][128 B u][4 + 4
        // scales] and then [128 B dg][128 B du].
        const int f0 = cur_ft * 256 + wg * 128;
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
          warp_rows();
          if (f0 < K) {
            uint8_t* dst = p.out + first * (2 * K) + f0;
            store_rows<128>(dst, 2 * K, slot0, valid, lane);
            store_rows<128>(dst + K, 2 * K, slot0 + 128u, valid, lane);
          }
          if (cur_row >= 0 && f0 < K) {
            const int64_t blk = f0 / 128;
            p.out_scales[blk * p.M + cur_row] = exp2_int(eg);
            p.out_scales[(blk + K / 128) * p.M + cur_row] = exp2_int(eu);
          }
        }
      } else {
        const int F = BWD ? p.K : p.N;
        const int f0 = cur_ft * 256 + wg * 128;
#pragma unroll
        for (int c = 0; c < 16; ++c)
          sts128(slot + 16u * c, pack_bf16x2(acc[8 * c], acc[8 * c + 1]),
                 pack_bf16x2(acc[8 * c + 2], acc[8 * c + 3]), pack_bf16x2(acc[8 * c + 4], acc[8 * c + 5]),
                 pack_bf16x2(acc[8 * c + 6], acc[8 * c + 7]));
        warp_rows();
        if (f0 < F)                          // F % 16 == 0: whole 32-byte pieces
          store_rows<256>(p.out + 2 * (first * F + f0), 2 * static_cast<int64_t>(F), slot0, valid, lane,
                          2u * static_cast<uint32_t>(min(128, F - f0)));
      }
      __syncwarp();                          // the slots have been read
      // (SwiGLU backward: the next rows come there by bulk copy)
      if constexpr (kGluBwd) fence_proxy_async_smem();
    }
  }

  tc_fence_before();
  __syncwarp();
  // A pair frees its tensor memory only when the even CTA's MMAs, which read
  // and write both CTAs, have drained and both epilogues are done.
  if constexpr (PAIR) cluster_sync_all(); else __syncthreads();
  tc_fence_after();
  // (the last of the commits that arrive in a pair's odd CTA)
  if (rank == 1 && threadIdx.x == 0) mbar_drain(drain_bar, 0);
  if (*abort_flag) {
    // A wait has run out, in this CTA or in the pair's other one, and every role
    // has stopped, each where it was: copies may be in flight for which nobody
    // has waited. They land before a CTA can exit.
    if (threadIdx.x == 0 && rank == 0) {
      const uint32_t mine = lds32(fills_at);
      uint32_t other = mine;
      if constexpr (PAIR)
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(other) : "r"(cluster_addr(fills_at, 1)) : "memory");
      FullBars8 b = {full(0), kStage8};
      close_fills(mine, other, S, b);
    }
    if (kGluBwd && threadIdx.x == 96) {
      const uint32_t n = lds32(ck_tiles_at);
      if (n > 0) mbar_drain(gu_bar, (n - 1) & 1u);
    }
    __syncwarp();
    if constexpr (PAIR) cluster_sync_all(); else __syncthreads();
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, 512); else tmem_dealloc(tmem_base, 512);
  }
}

template <int BWD, int EPI>
cudaError_t launch_fp8_gemm_t(const CUtensorMap& ta, const CUtensorMap& tw, const Fp8GemmArgs& p,
                              int form, int grid, cudaStream_t s) {
  const bool pair = form == kPair8;
  auto k = pair             ? grouped_fp8_gemm_kernel<BWD, EPI, kPair8>
           : form == kFew8  ? grouped_fp8_gemm_kernel<BWD, EPI, kFew8>
           : form == kSome8 ? grouped_fp8_gemm_kernel<BWD, EPI, kSome8>
                            : grouped_fp8_gemm_kernel<BWD, EPI, kSingle8>;
  const size_t smem = smem_bytes8(p.E, form);
  // (always to the same value, so that calls from several host threads agree)
  cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem_bytes8(1024, form)));
  if (err != cudaSuccess) return err;
  if (!pair) return launch_pdl(k, dim3(grid), dim3(kThreads8), smem, s, ta, tw, p);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads8);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  // Persistent pairs: as many as can be resident together (counted once per device).
  static std::atomic<int> max_pairs[64];
  int dev = 0;
  err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int n = max_pairs[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    cfg.numAttrs = 1;
    cfg.dynamicSmemBytes = smem_bytes8(1024, 1);
    err = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
    cfg.dynamicSmemBytes = smem;
    if (err != cudaSuccess) return err;
    if (n < 1) return cudaErrorInvalidConfiguration;
    max_pairs[dev].store(n, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3(std::min(grid, 2 * n));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, ta, tw, p);
}

}  // namespace

cudaError_t launch_grouped_fp8_gemm(bool bwd, int epi, const CUtensorMap& ta, const CUtensorMap& tw,
                                    const Fp8GemmArgs& p, int form, int grid, cudaStream_t s) {
  if (!bwd)
    return epi == MOE_EPI_SWIGLU ? launch_fp8_gemm_t<0, MOE_EPI_SWIGLU>(ta, tw, p, form, grid, s)
                                 : launch_fp8_gemm_t<0, MOE_EPI_NONE>(ta, tw, p, form, grid, s);
  return epi == MOE_EPI_SWIGLU_BWD ? launch_fp8_gemm_t<1, MOE_EPI_SWIGLU_BWD>(ta, tw, p, form, grid, s)
                                   : launch_fp8_gemm_t<1, MOE_EPI_NONE>(ta, tw, p, form, grid, s);
}

}  // namespace moeq
