// Scored routing (softmax or sigmoid scores, selection bias, expert groups,
// renormalised gates), its gradient, and the combine's backward that produces
// the gate gradient.
//
// The group tables and the row permutation are those of route.cu; only the
// selection differs. Definitions: include/moeq.h, moe_route_scored.
//
// A token's selection is a chain of dependent warp reductions (about 2 us),
// so what bounds it is latency: a warp per token, everything in registers,
// three launches for many tokens and one for a decode batch. Measured, whole
// call in a graph: 1 token of 384 experts in 8 groups with bias 9.7 us, 32
// tokens 15, 4096 tokens of 256 experts 21 to 25 (about 13 of it the scan of the
// counts and the scatter; 35 for k = 32), 16384 of 384 softmax without groups 40 (to
// read the 25 MB of logits would take 4). FP32 keys against 64-bit keys
// throughout: 39.5 / 88 us, and for the 4096 tokens, then in half as many
// blocks, 32.5 / 51. A token whose keys need 64 bits takes some 5 us more, and in a
// few thousand there are some, so the bound on the FP32 keys' error counts.
#include <algorithm>

#include "common.cuh"
#include "launchers.cuh"

namespace moeq {

namespace {

// 32 warps: two tokens each in large launches, one in small ones.
constexpr int kScoredThreads = 1024;
constexpr int kScoredWarps = kScoredThreads / 32;
constexpr int kScoredMaxSmem = 200 * 1024;

// False for NaN and -inf, which mask an expert.
__device__ __forceinline__ bool is_open(float l) { return l > -INFINITY; }

__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-static_cast<double>(l))); }

// Unsigned integers with the order of the floating numbers (no NaN; -0 is +0).
// Numbers map far above the two values kept for entries below every key.
constexpr uint32_t kKeyOut = 0u;      // not a candidate (taken, or of a closed group)
constexpr uint32_t kKeyMasked = 1u;   // a masked expert: chosen last, in ascending id
__device__ __forceinline__ uint32_t ordered_key(float v) {
  const int b = __float_as_int(v + 0.0f);
  return static_cast<uint32_t>(b) ^ (b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ unsigned long long ordered_key(double v) {
  const long long b = __double_as_longlong(v + 0.0);
  return static_cast<unsigned long long>(b) ^
         (b < 0 ? 0xffffffffffffffffull : 0x8000000000000000ull);
}

struct WarpBest {
  uint32_t hi, lo;   // the key (lo: low word of a 64-bit key, else 0)
  int idx;
};

// The warp's largest (key, then lowest id) of one candidate per lane, by
// integer warp reductions.
__device__ __forceinline__ WarpBest warp_best(uint32_t key, int idx) {
  const unsigned full = 0xffffffffu;
  WarpBest r;
  r.hi = __reduce_max_sync(full, key);
  r.lo = 0u;
  r.idx = static_cast<int>(__reduce_min_sync(full, key == r.hi ? static_cast<uint32_t>(idx) : 0x7fffffffu));
  return r;
}
__device__ __forceinline__ WarpBest warp_best(unsigned long long key, int idx) {
  const unsigned full = 0xffffffffu;
  const uint32_t hi = static_cast<uint32_t>(key >> 32), lo = static_cast<uint32_t>(key);
  WarpBest r;
  r.hi = __reduce_max_sync(full, hi);
  r.lo = __reduce_max_sync(full, hi == r.hi ? lo : 0u);
  r.idx = static_cast<int>(__reduce_min_sync(
      full, (hi == r.hi && lo == r.lo) ? static_cast<uint32_t>(idx) : 0x7fffffffu));
  return r;
}

// Elements from one group's values to the next in the warp's scratch: L lanes
// read a group, and a distance of L modulo 32 puts the 32 lanes' reads in
// distinct banks.
__host__ __device__ constexpr int group_lanes(int groups) {
  int P = 1;
  while (P < groups) P <<= 1;
  return 32 / P;
}
__host__ __device__ constexpr int group_pitch(int E, int groups) {
  const int gsize = E / groups;
  return gsize + ((group_lanes(groups) - gsize) & 31);
}

// e / gsize for e < 1024: the high word of e times ceil(2^32 / gsize) (an
// integer division takes some 20 instructions, and there are two an expert).
__device__ __forceinline__ uint32_t group_magic(int gsize) { return 0xffffffffu / static_cast<uint32_t>(gsize) + 1u; }
__device__ __forceinline__ int group_of(int e, uint32_t magic) {
  return magic == 0u ? e : static_cast<int>(__umulhi(static_cast<uint32_t>(e), magic));   // (0: one expert a group)
}

// Group scores and the open groups of one token, from the experts' values in
// gv (lane l: experts l + 32 i; -inf where masked) through the warp's row of
// shared memory. 32 / P lanes per group (P: groups rounded up to a power of
// two) each take every (32 / P)-th value and merge their two largest; lane g
// then holds group g's score, and a group stays open when fewer than
// topk_groups groups come before it. *gap: the distance between the last open
// and the first closed group's score.
template <typename Real, int NPER>
__device__ __forceinline__ unsigned open_groups(const Real (&gv)[NPER], Real* wrow, int E, const moe_router& rt,
                                                int lane, uint32_t magic, Real* gap) {
  const unsigned full = 0xffffffffu;
  const Real none = static_cast<Real>(-INFINITY);
  const int gsize = E / rt.groups;
  const int L = group_lanes(rt.groups), pitch = group_pitch(E, rt.groups);
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const int e = lane + 32 * i;
    if (e < E) wrow[e + group_of(e, magic) * (pitch - gsize)] = gv[i];
  }
  __syncwarp();
  const int g = lane / L;
  Real a = none, b = none;
  if (g < rt.groups) {
#pragma unroll 4
    for (int m = lane % L; m < gsize; m += L) {
      const Real v = wrow[g * pitch + m];
      b = fmax(b, fmin(a, v));
      a = fmax(a, v);
    }
  }
  for (int o = 1; o < L; o <<= 1) {
    const Real oa = __shfl_xor_sync(full, a, o), ob = __shfl_xor_sync(full, b, o);
    b = fmax(fmin(a, oa), fmax(b, ob));
    a = fmax(a, oa);
  }
  const Real mine = (rt.group_top == 2 && b > none) ? a + b : a;
  const Real gs = __shfl_sync(full, mine, min(lane, rt.groups - 1) * L);
  int before = 0;
  for (int o = 0; o < rt.groups; ++o) {
    const Real v = __shfl_sync(full, gs, o);
    before += (v > gs || (v == gs && o < lane)) ? 1 : 0;
  }
  const bool open = lane < rt.groups && before < rt.topk_groups;
  // Smallest open and largest closed score.
  Real lo_open = open ? gs : static_cast<Real>(INFINITY);
  Real hi_closed = (lane < rt.groups && !open) ? gs : none;
  for (int o = 16; o > 0; o >>= 1) {
    lo_open = fmin(lo_open, __shfl_xor_sync(full, lo_open, o));
    hi_closed = fmax(hi_closed, __shfl_xor_sync(full, hi_closed, o));
  }
  *gap = (rt.topk_groups < rt.groups) ? lo_open - hi_closed : static_cast<Real>(INFINITY);
  __syncwarp();
  return __ballot_sync(full, open);
}

// One token by one warp: lane j < k gets the j-th selected expert in my_idx,
// and whether it is unmasked in my_open; mx and total are the softmax's
// maximum and sum.
//
// Keys are compared as if in 64 bits. Without a bias the logits have the
// keys' order and are compared themselves, exactly. With a bias the keys are
// first formed in FP32. A sigmoid is off by less than 2^-21: with t = __expf(-l)
// (2 + 1.173 |l| ulp), s (1 - s) (2 + 1.173 |l|) 2^-23 <= 0.63 x 2^-23, the sum 1 + t
// 2^-24, __fdividef 2 ulp. A softmax score p is off by less than 2^-18 p, p <= 1 / z:
// expf 2 ulp and its argument's rounding in p and in z, a sum of positive
// numbers at most 37 additions deep, a quotient, a product. Adding the bias, or
// two keys of a group, rounds by 2^-24 of the sum, less than the 2^-22 allowed
// for it (top: the largest key). If every two neighbours of the sorted selection, the first one
// left out, and the groups around the cut lie further apart than twice that,
// the selection is the one in 64 bits. Where only neighbours are too close
// (one token in some hundreds for normal logits), the experts that may belong to
// the selection, at most 32, are ordered by their keys in 64 bits, one a lane;
// otherwise (groups too close, more than 32 candidates, masked experts
// reached) the whole token is done again in 64 bits.
template <int NPER>
__device__ __forceinline__ void select_token(const float* __restrict__ row, const float* __restrict__ bias, int E,
                                             int k, const moe_router& rt, double* wrow, int lane, float* mx_out,
                                             float* total_out, int* my_idx_out, bool* my_open_out) {
  const unsigned full = 0xffffffffu;
  const bool grouped = rt.groups > 1, softmax = rt.score == MOE_SCORE_SOFTMAX;
  const uint32_t magic = group_magic(E / rt.groups);
  float l[NPER], ez[NPER];              // logits (masked: -inf); softmax: exp(l - mx)
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const int e = lane + 32 * i;
    const float v = (e < E) ? __ldg(row + e) : -INFINITY;
    l[i] = is_open(v) ? v : -INFINITY;
    ez[i] = 0.0f;
    mx = fmaxf(mx, l[i]);
  }
  float z = 1.0f;
  if (softmax) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(full, mx, o));
    z = 0.0f;
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (is_open(l[i])) {
        ez[i] = (l[i] == mx) ? 1.0f : expf(l[i] - mx);
        z += ez[i];
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(full, z, o);
  }
  const float zinv = 1.0f / z;
  *mx_out = mx;
  *total_out = z;
  const bool scores = bias != nullptr || (grouped && rt.group_top == 2);   // else logits do for all
  int my_idx = 0;
  bool my_open = false, sure = true;
  {
    uint32_t key[NPER];
    float gv[NPER];
    float top = 0.0f;                     // largest magnitude of a key, for its error
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const int e = lane + 32 * i;
      float kv = l[i];
      gv[i] = l[i];
      if (scores && is_open(l[i])) {
        gv[i] = softmax ? ez[i] * zinv : __fdividef(1.0f, 1.0f + __expf(-l[i]));
        if (bias) {
          gv[i] += __ldg(bias + e);
          if (!(gv[i] > -INFINITY)) gv[i] = -INFINITY;
          kv = gv[i];
        }
        if (gv[i] > -INFINITY) top = fmaxf(top, fabsf(gv[i]));
      }
      key[i] = (e < E) ? ((kv > -INFINITY) ? ordered_key(kv) : kKeyMasked) : kKeyOut;
    }
    float err = 0.0f;
    if (scores) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(full, top, o));
      // 2^-18 / z or 2^-21, and 2^-22 top
      err = (softmax ? 3.814697265625e-6f * zinv : 4.76837158203125e-7f) + 2.384185791015625e-7f * top;
    }
    if (grouped) {
      float gap;
      const unsigned open = open_groups<float, NPER>(gv, reinterpret_cast<float*>(wrow), E, rt, lane, magic, &gap);
      // (a group score is one value or the sum of two)
      if (scores) sure = gap > 2.0f * rt.group_top * err;
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        const int e = lane + 32 * i;
        if (e < E && !((open >> group_of(e, magic)) & 1u)) key[i] = kKeyOut;
      }
    }
    // k rounds; with inexact keys more, while a key may still belong to the
    // selection (it is within reach of the k-th), and one for the first that
    // cannot. Lane j holds the j-th candidate; a 33rd, which no lane holds, is
    // still looked at: with one within reach, close keys need the whole token in 64 bits.
    // Each lane keeps its three best keys in order; a lane that has given all
    // three (rare: four of the selected experts in one lane) looks through its
    // keys again for those behind the last one it gave.
    uint32_t q0, q1, q2;
    int i0, i1, i2;
    auto refill = [&](uint32_t below, int after) {
      q0 = q1 = q2 = kKeyOut;
      i0 = i1 = i2 = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        const int e = lane + 32 * i;
        const uint32_t kx = (key[i] < below || (key[i] == below && e > after)) ? key[i] : kKeyOut;
        // (an equal key stays behind: ascending id)
        const bool u0 = kx > q0, u1 = kx > q1, u2 = kx > q2;
        q2 = u1 ? q1 : (u2 ? kx : q2);
        i2 = u1 ? i1 : (u2 ? e : i2);
        q1 = u0 ? q0 : (u1 ? kx : q1);
        i1 = u0 ? i0 : (u1 ? e : i1);
        q0 = u0 ? kx : q0;
        i0 = u0 ? e : i0;
      }
    };
    refill(0xffffffffu, 0x7fffffff);
    int given = 0;
    const int rounds = bias ? min(33, E) : k;
    float last = 0.0f, reach = 0.0f;
    int count = 0;
    bool close = false, odd = false;      // neighbours too close; only 64 bits will do
    for (int j = 0; j < rounds; ++j) {
      const WarpBest best = warp_best(q0, i0);
      if (bias) {
        const float v = __uint_as_float(best.hi ^ ((best.hi & 0x80000000u) ? 0x80000000u : 0xffffffffu));
        const bool real = best.hi > kKeyMasked;
        if (j >= k && !(real && v >= reach)) break;          // nothing more in reach
        odd |= !real;
        close |= j > 0 && !(last - v > 2.0f * err);
        last = v;
        if (j == k - 1) reach = v - 4.0f * err;
      }
      if (lane == j) {
        my_idx = best.idx;
        my_open = best.hi > kKeyMasked;
      }
      ++count;
      const bool gave = i0 == best.idx;
      if (gave) {
        q0 = q1;
        i0 = i1;
        q1 = q2;
        i1 = i2;
        q2 = kKeyOut;
        i2 = 0x7fffffff;
        ++given;
      }
      if (NPER > 3 && __any_sync(full, gave && given == 3)) {
        if (gave && given == 3) {
          refill(best.hi, best.idx);
          given = 0;
        }
      }
    }
    if (bias && (close || odd)) {
      if (odd || count > 32 || !(err < INFINITY)) {
        sure = false;
      } else if (sure) {
        // Order the candidates by their keys in 64 bits.
        double z64 = 1.0;
        if (softmax) {
          z64 = 0.0;
#pragma unroll
          for (int i = 0; i < NPER; ++i)
            if (is_open(l[i])) z64 += (l[i] == mx) ? 1.0 : exp(static_cast<double>(l[i]) - mx);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) z64 += __shfl_xor_sync(full, z64, o);
        }
        unsigned long long mine = kKeyOut;
        if (lane < count) {
          const float v = __ldg(row + my_idx);
          const double sv = softmax ? ((v == mx) ? 1.0 : exp(static_cast<double>(v) - mx)) / z64 : sigmoid64(v);
          mine = ordered_key(sv + static_cast<double>(__ldg(bias + my_idx)));
        }
        const int cand = my_idx;
        for (int j = 0; j < k; ++j) {
          const WarpBest best = warp_best(mine, lane < count ? cand : 0x7fffffff);
          if (lane == j) my_idx = best.idx;
          if (lane < count && cand == best.idx) mine = kKeyOut;
        }
        my_open = lane < k;
      }
    }
  }
  if (scores && !__all_sync(full, sure)) {
    // In 64 bits.
    double z64 = 1.0;
    if (softmax) {
      z64 = 0.0;
#pragma unroll
      for (int i = 0; i < NPER; ++i)
        if (is_open(l[i])) z64 += (l[i] == mx) ? 1.0 : exp(static_cast<double>(l[i]) - mx);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z64 += __shfl_xor_sync(full, z64, o);
      *total_out = static_cast<float>(z64);
    }
    unsigned long long key[NPER];
    double gv[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const int e = lane + 32 * i;
      double kv = l[i];
      gv[i] = l[i];
      if (is_open(l[i])) {
        gv[i] = softmax ? ((l[i] == mx) ? 1.0 : exp(static_cast<double>(l[i]) - mx)) / z64 : sigmoid64(l[i]);
        if (bias) {
          gv[i] += static_cast<double>(__ldg(bias + e));
          if (!(gv[i] > -INFINITY)) gv[i] = -INFINITY;
          kv = gv[i];
        }
      }
      key[i] = (e < E) ? ((kv > -INFINITY) ? ordered_key(kv) : kKeyMasked) : kKeyOut;
    }
    if (grouped) {
      double gap;
      const unsigned open = open_groups<double, NPER>(gv, wrow, E, rt, lane, magic, &gap);
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        const int e = lane + 32 * i;
        if (e < E && !((open >> group_of(e, magic)) & 1u)) key[i] = kKeyOut;
      }
    }
    for (int j = 0; j < k; ++j) {
      unsigned long long bk = kKeyOut;
      int bi = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < NPER; ++i)
        if (key[i] > bk) {
          bk = key[i];
          bi = lane + 32 * i;
        }
      const WarpBest best = warp_best(bk, bi);
      if (lane == j) {
        my_idx = best.idx;
        my_open = best.hi != 0u;
      }
#pragma unroll
      for (int i = 0; i < NPER; ++i)
        if (lane + 32 * i == best.idx) key[i] = kKeyOut;
    }
  }
  *my_idx_out = my_idx;
  *my_open_out = my_open && lane < k;
}

// exp(v - ref) for v <= ref, to a few ulp: the rounding of the difference, up
// to 2^-18 of the result by itself, is put back.
__device__ __forceinline__ float exp_below(float v, float ref) {
  if (v == ref) return 1.0f;              // (two infinities too)
  const float d = v - ref;
  if (!(d > -110.0f)) return 0.0f;        // below FP32's smallest
  const float back = d - v;
  const float rest = (v - (d - back)) - (ref + back);   // v - ref - d, exactly
  const float s = expf(d);
  return fmaf(s, rest, s);
}

// Gate of the lane's selected expert, in FP32. With renorm a softmax is taken
// over the selected logits alone, which is the same quotient without the small
// numbers (a bias or closed groups can leave only scores far below the largest);
// sigmoids far below zero, whose quotients FP32 does not hold, are taken in 64 bits.
__device__ __forceinline__ float gate_of(const float* __restrict__ row, int idx, bool open, float mx, float total,
                                         const moe_router& rt) {
  const unsigned full = 0xffffffffu;
  const bool softmax = rt.score == MOE_SCORE_SOFTMAX;
  const float v = open ? __ldg(row + idx) : -INFINITY;
  float s = 0.0f;
  if (!rt.renorm) {
    if (open) s = softmax ? exp_below(v, mx) / total : 1.0f / (1.0f + expf(-v));
    return rt.scale * s;
  }
  if (softmax) {
    float top = v;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(full, top, o));
    // (scores that are 0 in 64 bits sum to 0)
    if (open && (top == mx || exp(static_cast<double>(top) - mx) > 0.0)) s = exp_below(v, top);
  } else if (open) {
    s = 1.0f / (1.0f + expf(-v));
  }
  if (softmax || !__any_sync(full, open && v < -64.0f)) {
    float sum = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(full, sum, o);
    return rt.scale * (sum > 0.0f ? s / sum : 0.0f);
  }
  const double s64 = open ? sigmoid64(v) : 0.0;
  double sum64 = s64;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum64 += __shfl_xor_sync(full, sum64, o);
  return static_cast<float>(rt.scale * (sum64 > 0.0 ? s64 / sum64 : 0.0));
}

// tpb tokens per block, or per cluster of two blocks (parts = 2), which add
// their histograms; block_counts == nullptr skips the histogram.
template <int NPER>
__global__ void __launch_bounds__(kScoredThreads, 1)
route_scored_kernel(const float* __restrict__ logits, const float* __restrict__ bias, int T, int E, int k, int tpb,
                    int parts, int row_el, moe_router rt, int32_t* __restrict__ topk_idx, float* __restrict__ gates,
                    int32_t* __restrict__ block_counts) {
  extern __shared__ double scored_sm[];   // [warps][row_el] group scratch; then [E] histogram
  grid_dependency_wait();
  grid_dependents_launch();
  const int warps = blockDim.x >> 5;
  int32_t* hist = reinterpret_cast<int32_t*>(scored_sm + warps * row_el);
  const bool with_hist = block_counts != nullptr;
  if (with_hist)
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = parts == 2 ? static_cast<int>(cluster_ctarank()) : 0;
  const int group = static_cast<int>(blockIdx.x) / parts, mine = tpb / parts;
  for (int u = warp; u < mine; u += warps) {
    const int t = group * tpb + rank * mine + u;
    if (t >= T) break;
    const float* row = logits + static_cast<int64_t>(t) * E;
    float mx;
    float total;
    int idx;
    bool open;
    select_token<NPER>(row, bias, E, k, rt, scored_sm + warp * row_el, lane, &mx, &total, &idx,
                       &open);
    const float w = gate_of(row, idx, open, mx, total, rt);
    if (lane < k) {
      topk_idx[static_cast<int64_t>(t) * k + lane] = idx;
      gates[static_cast<int64_t>(t) * k + lane] = w;
      if (with_hist) atomicAdd(&hist[idx], 1);
    }
  }
  if (!with_hist) return;
  if (parts == 2) cluster_sync_all(); else __syncthreads();
  if (rank == 0)
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      int32_t n = hist[e];
      if (parts == 2) {
        int32_t other;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(other) : "r"(cluster_addr(smem_u32(&hist[e]), 1)) : "memory");
        n += other;
      }
      block_counts[static_cast<int64_t>(group) * E + e] = n;
    }
  if (parts == 2) cluster_sync_all();     // (the other block's counts have been read)
}

// Up to 32 tokens (a decode batch) in one block and one launch: a warp per
// token selects, then the block forms the group tables and the permutation
// from one 32-bit token mask per expert.
constexpr int kSmallTokens = 32;
template <int NPER>
__global__ void __launch_bounds__(kScoredThreads, 1)
route_scored_small_kernel(const float* __restrict__ logits, const float* __restrict__ bias, int T, int E, int k,
                          int row_el, moe_router rt, int chunk_size, int32_t* __restrict__ topk_idx, float* __restrict__ gates,
                          int32_t* __restrict__ offsets, int32_t* __restrict__ active,
                          int32_t* __restrict__ num_active, int32_t* __restrict__ chunk_offsets,
                          int32_t* __restrict__ num_chunks, int32_t* __restrict__ perm_token,
                          int32_t* __restrict__ inv_perm) {
  extern __shared__ double scored_sm[];   // [T][row_el] group scratch
  __shared__ uint32_t mask[1024];
  __shared__ int32_t first[1024];
  __shared__ int32_t chosen[kSmallTokens * 32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  mask[tid] = 0u;
  __syncthreads();
  if (warp < T) {
    const float* row = logits + static_cast<int64_t>(warp) * E;
    float mx;
    float total;
    int idx;
    bool open;
    select_token<NPER>(row, bias, E, k, rt, scored_sm + warp * row_el, lane, &mx, &total, &idx,
                       &open);
    if (lane < k) {
      chosen[warp * k + lane] = idx;
      atomicOr(&mask[idx], 1u << warp);
      topk_idx[warp * k + lane] = idx;
    }
    const float w = gate_of(row, idx, open, mx, total, rt);
    if (lane < k) gates[warp * k + lane] = w;
  }
  __syncthreads();
  first[tid] = scan_experts(tid < E ? __popc(mask[tid]) : 0, E, chunk_size, offsets, active, num_active,
                            chunk_offsets, num_chunks);
  __syncthreads();
  if (tid < T * k) {
    const int t = tid / k, e = chosen[tid];
    const int p = first[e] + __popc(mask[e] & ((1u << t) - 1u));
    perm_token[p] = t;
    inv_perm[tid] = p;
  }
}

// One warp per token: the k selected experts' ds in the lanes, spread into a
// row of the warp's shared memory, then the whole row of d_logits written
// once. What belongs to the k selected scores is in 64 bits, because renorm
// subtracts nearly equal numbers and divides by a sum that may lie below
// FP32; the dense softmax part is in 32. Bound: latency, not the one row of
// logits read (softmax) and one of d_logits written: a warp makes up to three
// passes over the row with 4-byte accesses, and the 64-bit exponentials keep k of
// 32 lanes busy. 4096 x 384: softmax 10.7 us (13 MB, 2.0 at the copy rate), sigmoid
// 5.1 (6.8 MB, 1.0), at 7 and 5 % of DRAM's throughput; 16384 x 384: 21.3 and 10.2.
constexpr int kBwdWarps = 8;
__global__ void __launch_bounds__(kBwdWarps * 32)
route_scored_bwd_kernel(const float* __restrict__ d_gates, const float* __restrict__ gates,
                        const float* __restrict__ logits, const int32_t* __restrict__ topk_idx, int T, int E,
                        int k, moe_router rt, float* __restrict__ d_logits) {
  extern __shared__ float bwd_sm[];     // [warps][E]
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned full = 0xffffffffu;
  const int t = blockIdx.x * kBwdWarps + warp;
  if (t >= T) return;
  float* ds_row = bwd_sm + warp * E;
  const float* row = logits + static_cast<int64_t>(t) * E;
  float* out = d_logits + static_cast<int64_t>(t) * E;
  const bool softmax = rt.score == MOE_SCORE_SOFTMAX;
  float mx = -INFINITY, total = softmax ? 0.0f : 1.0f;
  if (softmax) {
    for (int e = lane; e < E; e += 32) {
      const float v = __ldg(row + e);
      if (is_open(v)) mx = fmaxf(mx, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(full, mx, o));
  }
  if (softmax) {
    for (int e = lane; e < E; e += 32) {
      const float v = __ldg(row + e);
      if (is_open(v)) total += (v == mx) ? 1.0f : expf(v - mx);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(full, total, o);
  }
  int idx = -1;
  double dw = 0.0, s = 0.0, rest = 0.0;   // rest: 1 - s of the sigmoid, without cancellation
  if (lane < k) {
    idx = __ldg(topk_idx + static_cast<int64_t>(t) * k + lane);
    float v = (idx >= 0 && idx < E) ? __ldg(row + idx) : -INFINITY;
    if (gates && __ldg(gates + static_cast<int64_t>(t) * k + lane) == 0.0f) v = -INFINITY;   // masked in the forward
    if (is_open(v)) {
      dw = static_cast<double>(rt.scale) * __ldg(d_gates + static_cast<int64_t>(t) * k + lane);
      if (softmax) {
        s = ((v == mx) ? 1.0 : exp(static_cast<double>(v) - mx)) / total;
      } else {
        s = sigmoid64(v);
        rest = 1.0 / (1.0 + exp(static_cast<double>(v)));
      }
    } else {
      idx = -1;
    }
  }
  double sum = s, dot = dw * s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(full, sum, o);
    dot += __shfl_xor_sync(full, dot, o);
  }
  double ds = dw, back = dot;           // back: sum_j ds_j s_j of the softmax
  if (rt.renorm) {
    ds = sum > 0.0 ? (dw - dot / sum) / sum : 0.0;
    back = 0.0;                         // the gates do not change when every score is scaled
  }
  const float base = static_cast<float>(-back) / total;
  for (int e = lane; e < E; e += 32) {
    float g = 0.0f;
    if (softmax && !rt.renorm) {
      const float v = __ldg(row + e);
      if (is_open(v)) g = ((v == mx) ? 1.0f : expf(v - mx)) * base;
    }
    ds_row[e] = g;
  }
  __syncwarp();
  if (idx >= 0) ds_row[idx] = static_cast<float>(softmax ? s * (ds - back) : ds * s * rest);
  __syncwarp();
  for (int e = lane; e < E; e += 32) out[e] = ds_row[e];
}

}  // namespace

cudaError_t launch_route_scored(const float* logits, const float* bias, const void* x, int T, int E,
                                int k, int64_t d, const moe_router& rt, int chunk_size,
                                int32_t* topk_idx, float* gates, int32_t* offsets, int32_t* active,
                                int32_t* num_active, int32_t* chunk_offsets, int32_t* num_chunks,
                                int32_t* perm_token, int32_t* inv_perm, void* x_perm,
                                int32_t* block_counts, cudaStream_t s) {
  const int nper = (E + 31) / 32;
  // Selects the instantiation and raises its shared-memory limit, past 48 KiB
  // (more than 192 experts in groups).
#define MOEQ_BY_NPER(CALL_)             \
  (nper <= 2 ? CALL_(2)                 \
   : nper <= 4 ? CALL_(4)               \
   : nper <= 8 ? CALL_(8)               \
   : nper <= 12 ? CALL_(12)             \
   : nper <= 16 ? CALL_(16) : CALL_(32))
  // (always to the same value, so that calls from several host threads agree)
  auto go = [&](auto kern, int blocks, int threads, int parts, size_t sm, auto... args) {
    if (sm > 32 * 1024) {
      const cudaError_t e =
          cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kScoredMaxSmem);
      if (e != cudaSuccess) return e;
    }
    if (parts == 1) return launch_pdl(kern, dim3(blocks), dim3(threads), sm, s, args...);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = sm;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, args...);
  };
  // one warp's group scratch, in doubles
  const int row_el = rt.groups > 1 ? group_pitch(E, rt.groups) * rt.groups : 0;
  const size_t row_sm = sizeof(double) * row_el;
  // Warps of a block whose scratch fits (32, or 12 for the most padded groups).
  const int fit = row_sm == 0 ? kScoredWarps
                              : static_cast<int>(std::min<size_t>(kScoredWarps, (kScoredMaxSmem - 4096) / row_sm));
  if (T <= std::min(kSmallTokens, fit) && x == nullptr) {
#define MOEQ_SMALL(N_)                                                                                             \
  go(route_scored_small_kernel<N_>, 1, kScoredThreads, 1, row_sm* T, logits, bias, T, E, k, row_el, rt, chunk_size, topk_idx, gates, \
     offsets, active, num_active, chunk_offsets, num_chunks, perm_token, inv_perm)
    return MOEQ_BY_NPER(MOEQ_SMALL);
#undef MOEQ_SMALL
  }
  const bool small = route_single_pass(T, E);
  if (!small && block_counts == nullptr) return cudaErrorInvalidValue;
  const int tpb = small ? fit : route_tokens_per_block();
  const int nblk = static_cast<int>(blocks_for(T, tpb));
  int32_t* hist_out = small ? nullptr : block_counts;
  // Two blocks (a cluster, one token a warp instead of two) per histogram while
  // all of them can run at once, which halves the selection's share; above
  // that the cluster only costs. Measured (one / two blocks, us): 2048 tokens of
  // 256 experts in groups 33.2 / 24.7, 4096 33.5 / 26.0, 8192 35.0 / 37.2; 6000 of
  // 384 without groups 25.1 / 28.4, 16384 41.9 / 50.0.
  int sms = 0;
  cudaError_t err = route_prepare_device(&sms);
  if (err != cudaSuccess) return err;
  const int parts = !small && 2 * nblk <= sms ? 2 : 1;
  const size_t sm = row_sm * fit + (small ? 0 : sizeof(int32_t) * E);
#define MOEQ_LARGE(N_) \
  go(route_scored_kernel<N_>, nblk * parts, 32 * fit, parts, sm, logits, bias, T, E, k, tpb, parts, row_el, rt, topk_idx, gates, hist_out)
  err = MOEQ_BY_NPER(MOEQ_LARGE);
#undef MOEQ_LARGE
#undef MOEQ_BY_NPER
  if (err != cudaSuccess) return err;
  return launch_route_tables(x, T, E, k, d, chunk_size, topk_idx, offsets, active, num_active,
                             chunk_offsets, num_chunks, perm_token, inv_perm, x_perm, block_counts,
                             s);
}

cudaError_t launch_route_scored_bwd(const float* d_gates, const float* gates, const float* logits,
                                    const int32_t* topk_idx, int T, int E, int k,
                                    const moe_router& rt, float* d_logits, cudaStream_t s) {
  return launch_pdl(route_scored_bwd_kernel, dim3(blocks_for(T, kBwdWarps)),
                    dim3(kBwdWarps * 32), sizeof(float) * kBwdWarps * E, s, d_gates, gates, logits, topk_idx,
                    T, E, k, rt, d_logits);
}

}  // namespace moeq
