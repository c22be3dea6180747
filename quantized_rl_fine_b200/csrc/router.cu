// Scored routing (softmax or sigmoid scores, selection bias, expert groups,
// renormalised gates), its gradient, and the combine's backward that produces
// the gate gradient.
//
// The group tables and the row permutation are those of route.cu; only the
// selection differs. Definitions: include/moeq.h, moe_route_scored.
#include <algorithm>

#include "common.cuh"
#include "launchers.cuh"

namespace moeq {

namespace {

constexpr int kScoredThreads = 512;   // 16 warps, four tokens each in large launches
constexpr int kScoredWarps = kScoredThreads / 32;

// Unsigned integer with the order of the doubles (no NaN; -0 is +0). Real
// values map to at least 2^52 - 1, which leaves 0 and 1 for the two kinds of
// entry below every key.
constexpr unsigned long long kKeyOut = 0ull;      // not a candidate (taken, or of a closed group)
constexpr unsigned long long kKeyMasked = 1ull;   // a masked expert: chosen last, in ascending id
__device__ __forceinline__ unsigned long long ordered_key(double v) {
  const long long b = __double_as_longlong(v + 0.0);
  return static_cast<unsigned long long>(b) ^
         (b < 0 ? 0xffffffffffffffffull : 0x8000000000000000ull);
}

// False for NaN and -inf, which mask an expert.
__device__ __forceinline__ bool is_open(float l) { return l > -INFINITY; }

__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-static_cast<double>(l))); }

// One warp per token. Without a bias the logits themselves order the experts;
// KEYS64: scores are needed in 64 bits, for biased keys or for group sums.
// Each selection step takes the warp's largest 64-bit key with three integer
// warp reductions (high word, low word, lowest id), so ties need no shuffles.
template <int NPER, bool KEYS64>
__global__ void __launch_bounds__(kScoredThreads)
route_scored_kernel(const float* __restrict__ logits, const float* __restrict__ bias, int T, int E,
                    int k, int tpb, moe_router rt, int32_t* __restrict__ topk_idx,
                    float* __restrict__ gates, int32_t* __restrict__ block_counts) {
  extern __shared__ double scored_sm[];   // groups > 1: [warps][E] keys; then [E] histogram
  grid_dependency_wait();
  grid_dependents_launch();
  const bool grouped = rt.groups > 1;
  int32_t* hist = reinterpret_cast<int32_t*>(scored_sm + (grouped ? kScoredWarps * E : 0));
  const bool with_hist = block_counts != nullptr;
  if (with_hist)
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned full = 0xffffffffu;
  const int per_warp = tpb / kScoredWarps;
  double* wkeys = scored_sm + static_cast<int64_t>(warp) * E;
  const int gsize = E / rt.groups;
  const bool softmax = rt.score == MOE_SCORE_SOFTMAX;
  for (int u = 0; u < per_warp; ++u) {
    const int t = blockIdx.x * tpb + warp * per_warp + u;
    if (t >= T) break;
    const float* row = logits + static_cast<int64_t>(t) * E;
    float l[NPER];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const int e = lane + 32 * i;
      const float v = (e < E) ? __ldg(row + e) : -INFINITY;
      l[i] = is_open(v) ? v : -INFINITY;
      mx = fmaxf(mx, l[i]);
    }
    double total = 1.0;                  // softmax: sum of exp(l - mx)
    if (softmax) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(full, mx, o));
      if constexpr (KEYS64) {
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
          if (is_open(l[i])) z += (l[i] == mx) ? 1.0 : exp(static_cast<double>(l[i]) - mx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(full, z, o);
        total = z;
      } else {
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
          if (is_open(l[i])) z += (l[i] == mx) ? 1.0f : expf(l[i] - mx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(full, z, o);
        total = z;
      }
    }
    // Score of an expert with an unmasked logit (+inf included).
    auto score64 = [&](float v) {
      if (softmax) return ((v == mx) ? 1.0 : exp(static_cast<double>(v) - mx)) / total;
      return sigmoid64(v);
    };
    unsigned long long key[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const int e = lane + 32 * i;
      key[i] = kKeyOut;
      if (e >= E) continue;
      // kv orders the experts, gv is what groups add up.
      double kv = -INFINITY, gv = -INFINITY;
      if (is_open(l[i])) {
        kv = gv = static_cast<double>(l[i]);
        if constexpr (KEYS64) {
          gv = score64(l[i]);
          if (bias) {
            gv += static_cast<double>(__ldg(bias + e));
            kv = gv = (gv > -INFINITY) ? gv : -INFINITY;
          }
        }
      }
      key[i] = (kv > -INFINITY) ? ordered_key(kv) : kKeyMasked;
      if (grouped) wkeys[e] = gv;
    }
    if (grouped) {
      // 32 / P lanes per group (P: groups rounded up to a power of two) each
      // take every (32 / P)-th key of the group and merge their two largest.
      __syncwarp();
      int P = 1;
      while (P < rt.groups) P <<= 1;
      const int L = 32 / P;
      const int g = lane / L, sub = lane % L;
      double a = -INFINITY, b = -INFINITY;
      if (g < rt.groups) {
        for (int m = sub; m < gsize; m += L) {
          const double v = wkeys[g * gsize + m];
          if (v > a) { b = a; a = v; } else if (v > b) { b = v; }
        }
      }
      for (int o = 1; o < L; o <<= 1) {
        const double oa = __shfl_xor_sync(full, a, o), ob = __shfl_xor_sync(full, b, o);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
      }
      const double mine = (rt.group_top == 2 && b > -INFINITY) ? a + b : a;
      // Lane g holds group g; a group stays open when fewer than topk_groups
      // groups come before it.
      const double gs = __shfl_sync(full, mine, min(lane, rt.groups - 1) * L);
      int before = 0;
      for (int o = 0; o < rt.groups; ++o) {
        const double v = __shfl_sync(full, gs, o);
        before += (v > gs || (v == gs && o < lane)) ? 1 : 0;
      }
      const unsigned open = __ballot_sync(full, lane < rt.groups && before < rt.topk_groups);
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        const int e = lane + 32 * i;
        if (e < E && !((open >> (e / gsize)) & 1u)) key[i] = kKeyOut;
      }
      __syncwarp();
    }
    // k rounds of the warp's best key.
    unsigned long long bk = kKeyOut;
    int bi = 0x7fffffff;
    auto local_best = [&]() {
      bk = kKeyOut;
      bi = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < NPER; ++i)
        if (key[i] > bk) {
          bk = key[i];
          bi = lane + 32 * i;
        }
    };
    local_best();
    int my_idx = 0;
    bool my_open = false;
    for (int j = 0; j < k; ++j) {
      const unsigned hi = static_cast<unsigned>(bk >> 32), lo = static_cast<unsigned>(bk);
      const unsigned mh = __reduce_max_sync(full, hi);
      const unsigned ml = __reduce_max_sync(full, hi == mh ? lo : 0u);
      const int best = static_cast<int>(
          __reduce_min_sync(full, (hi == mh && lo == ml) ? static_cast<unsigned>(bi) : 0x7fffffffu));
      if (lane == j) {
        my_idx = best;
        my_open = mh != 0u;
      }
      if ((best & 31) == lane) {
#pragma unroll
        for (int i = 0; i < NPER; ++i)
          if (i == (best >> 5)) key[i] = kKeyOut;
        local_best();
      }
    }
    // The k selected scores in 64 bits: with renorm even scores that FP32
    // cannot hold (a sigmoid far below zero) give their gates.
    const double s = (lane < k && my_open) ? score64(__ldg(row + my_idx)) : 0.0;
    double sum = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(full, sum, o);
    if (lane < k) {
      const double w = rt.renorm ? (sum > 0.0 ? s / sum : 0.0) : s;
      topk_idx[static_cast<int64_t>(t) * k + lane] = my_idx;
      gates[static_cast<int64_t>(t) * k + lane] = static_cast<float>(rt.scale * w);
      if (with_hist) atomicAdd(&hist[my_idx], 1);
    }
  }
  if (!with_hist) return;
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x)
    block_counts[static_cast<int64_t>(blockIdx.x) * E + e] = hist[e];
}

// One warp per token: the k selected experts' ds in the lanes, spread into a
// row of the warp's shared memory, then the whole row of d_logits written
// once. What belongs to the k selected scores is in 64 bits, because renorm
// subtracts nearly equal numbers and divides by a sum that may lie below
// FP32; the dense softmax part is in 32.
constexpr int kBwdWarps = 8;
__global__ void __launch_bounds__(kBwdWarps * 32)
route_scored_bwd_kernel(const float* __restrict__ d_gates, const float* __restrict__ logits,
                        const int32_t* __restrict__ topk_idx, int T, int E, int k, moe_router rt,
                        float* __restrict__ d_logits) {
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
    const float v = (idx >= 0 && idx < E) ? __ldg(row + idx) : -INFINITY;
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
  const bool small = route_single_pass(T, E);
  if (!small && block_counts == nullptr) return cudaErrorInvalidValue;
  const int tpb = small ? kScoredWarps : route_tokens_per_block();
  const int nblk = (T + tpb - 1) / tpb;
  int32_t* hist_out = small ? nullptr : block_counts;
  const size_t sm = (rt.groups > 1 ? sizeof(double) * kScoredWarps * E : 0) +
                    (small ? 0 : sizeof(int32_t) * E);
  const bool keys64 = bias != nullptr || (rt.groups > 1 && rt.group_top == 2);
  const int nper = (E + 31) / 32;
  cudaError_t err;
  // The shared-memory limit only matters past 48 KiB (more than 384 experts in groups).
#define MOEQ_SCORED_T(N_, K_)                                                                       \
  [&]() {                                                                                           \
    if (sm > 48 * 1024) {                                                                           \
      const cudaError_t e_ = cudaFuncSetAttribute(                                                  \
          route_scored_kernel<N_, K_>, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);    \
      if (e_ != cudaSuccess) return e_;                                                             \
    }                                                                                               \
    return launch_pdl(route_scored_kernel<N_, K_>, dim3(nblk), dim3(kScoredThreads), sm, s, logits, \
                      bias, T, E, k, tpb, rt, topk_idx, gates, hist_out);                           \
  }()
#define MOEQ_SCORED(N_) (keys64 ? MOEQ_SCORED_T(N_, true) : MOEQ_SCORED_T(N_, false))
  if (nper <= 2) err = MOEQ_SCORED(2);
  else if (nper <= 4) err = MOEQ_SCORED(4);
  else if (nper <= 8) err = MOEQ_SCORED(8);
  else if (nper <= 12) err = MOEQ_SCORED(12);
  else if (nper <= 16) err = MOEQ_SCORED(16);
  else err = MOEQ_SCORED(32);
#undef MOEQ_SCORED
#undef MOEQ_SCORED_T
  if (err != cudaSuccess) return err;
  return launch_route_tables(x, T, E, k, d, chunk_size, topk_idx, offsets, active, num_active,
                             chunk_offsets, num_chunks, perm_token, inv_perm, x_perm, block_counts,
                             s);
}

cudaError_t launch_route_scored_bwd(const float* d_gates, const float* logits,
                                    const int32_t* topk_idx, int T, int E, int k,
                                    const moe_router& rt, float* d_logits, cudaStream_t s) {
  return launch_pdl(route_scored_bwd_kernel, dim3((T + kBwdWarps - 1) / kBwdWarps),
                    dim3(kBwdWarps * 32), sizeof(float) * kBwdWarps * E, s, d_gates, logits, topk_idx,
                    T, E, k, rt, d_logits);
}

}  // namespace moeq
