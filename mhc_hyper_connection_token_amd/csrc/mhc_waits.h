// mhc_waits.h -- how many direct loads into LDS a wave of the staged dots
// (mhc_pre_bwd.hip) may leave in flight when it turns to a unit of work.  Plain C++,
// so that the counts can be checked against the order of the requests without a GPU.
#pragma once

namespace mhc {

constexpr int kDyLoads = 4;  // a wave's loads of dy a slice

// Three stages.  A wave asks for dy of the first slice, unit 0 and unit 1 (`unit_loads`
// each) and then, in unit u, for dy of the next slice if unit u begins one (stream 0)
// and for unit u + 2; loads land in the order of the requests.  Turning to unit u of
// stream c, unit u must have landed and unit u + 1 may be on its way, with the four of
// dy between the two where unit u - 1 began a slice.  Unit u - 1 + S reads that dy: with
// one stream that is unit u itself, and dy has to have landed too.
constexpr int dots_in_flight(int streams, int c, int unit_loads) {
  return unit_loads + (streams > 1 && c == 1 ? kDyLoads : 0);
}

}  // namespace mhc
