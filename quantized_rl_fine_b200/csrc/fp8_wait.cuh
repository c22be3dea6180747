// How the FP8 product's waits measure their budget, and how a CTA or pair
// whose waits have run out brings its copies to an end, in plain arithmetic
// that also compiles for the host.
#pragma once

#include <stdint.h>

namespace moeq {

// Waits count time in units of 1024 cycles, held in 32 bits (the epilogue has
// no registers for more); differences are taken modulo 2^32 units.
constexpr int kWaitUnitBits = 10;
// The longest budget: half the range of the count, 2^41 cycles (20 minutes),
// so that a waiting thread, which looks at least every 0.2 ms, cannot miss it.
constexpr uint32_t kMaxWaitUnits = 1u << 31;

__host__ __device__ constexpr uint32_t wait_units(long long clock) {
  return static_cast<uint32_t>(static_cast<unsigned long long>(clock) >> kWaitUnitBits);
}

// Whether a wait that began at unit t0 has used up `budget` cycles at unit
// now: never before, and at most three units after (two for the two clocks'
// positions inside a unit, one for the budget's).
__host__ __device__ constexpr bool wait_spent(uint32_t t0, uint32_t now, long long budget) {
  const unsigned long long units = static_cast<unsigned long long>(budget) >> kWaitUnitBits;
  const uint32_t limit = units < kMaxWaitUnits ? static_cast<uint32_t>(units) : kMaxWaitUnits;
  return now - t0 > limit + 1u;
}

// Waits for the copies of the fills that nobody has waited for, once no role
// begins another. Fill g goes to stage g % stages and completes phase
// g / stages of that stage's barrier, which lies in the CTA that calls this:
// one arrival, by this CTA, and both CTAs' bytes in a pair. `mine` and `other`
// are the fills that this CTA and the pair's other one have begun (equal for a
// CTA alone). They differ by `stages` at most, because a stage is filled again
// only after its fill by both has been used. Where one CTA has gone further,
// what the other would have added is supplied first:
//   bars.add_bytes(stage)   the other CTA's bytes of a fill, which will not come
//   bars.arrive(stage)      this CTA's arrival for a fill of the other one's bytes alone
//   bars.wait(stage, parity)
template <class Bars>
__host__ __device__ inline void close_fills(uint32_t mine, uint32_t other, uint32_t stages, Bars& bars) {
  for (uint32_t g = other; g < mine; ++g) bars.add_bytes(g % stages);
  for (uint32_t g = mine; g < other; ++g) bars.arrive(g % stages);
  const uint32_t end = mine > other ? mine : other;
  for (uint32_t g = end > stages ? end - stages : 0u; g < end; ++g) bars.wait(g % stages, (g / stages) & 1u);
}

}  // namespace moeq
