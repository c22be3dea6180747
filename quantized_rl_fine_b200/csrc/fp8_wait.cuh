// How the FP8 product's waits measure their budget, in plain arithmetic that
// also compiles for the host.
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

}  // namespace moeq
