// Where the two softmax groups of the tcgen05 tree attention leave each other their rows' (maximum,
// sum) at the end of a unit of up to 128 rows.
//
// A group writes its own, both arrive at the barrier `met` of the unit, and both read both. A group
// that has a step in the next unit waits there for the other one (scores need the queries that both
// have stored after reading); with a single tile in it, the second group has none and comes to its
// next write with nothing but its own work behind it, while the first may still be reading. So
// units take turns between two places: a group writes the place of unit u again in unit u + 2, after
// `met` of unit u + 1, at which the other arrives when it has read unit u's.
#pragma once

namespace pkv {

constexpr int kExchangeRows = 128;
constexpr int kExchangeSlots = 2 * 2 * kExchangeRows;

#ifdef __CUDACC__
__host__ __device__
#endif
constexpr int exchange_slot(unsigned unit, int group, int row) {
  return (int)((unit & 1u) * 2u + (unsigned)group) * kExchangeRows + row;
}

}  // namespace pkv
