// Host-only check of the lanes of a head's row, built with g++ and its sanitizers by
// tests/test_host_lanes.py: over every length and rotation the most that the kernels
// are built for is not exceeded, and is reached, so that none is built for nothing.
// Prints "ALL OK" and exits 0 when every check holds.
#include <cstdio>
#include <map>
#include <tuple>

#include "../../newton_schulz_05_amd/csrc/ops_limits.hpp"

using namespace muon;

int main() {
  std::map<std::tuple<bool, bool, int>, int> most;
  int bad = 0;
  for (int size : {2, 4})
    for (int dim = 1; dim <= kHeadMaxDim; ++dim)
      for (int rot = 0; rot <= dim; rot += 2)
        for (bool inter : {false, true}) {
          const int piece = 16 / size, half = rot / 2;
          const bool whole = inter ? dim % piece == 0 && half % (piece / 2) == 0
                                   : half % piece == 0 && (dim - rot) % piece == 0;
          const int lanes = head_lanes(dim, rot, inter);
          int& m = most[{inter, whole, size}];
          m = lanes > m ? lanes : m;
          // every element has a place
          const int held = inter || rot == 0 ? lanes * 16 : 16 * ((half + 7) / 8) + 16 * (lanes - (half + 7) / 8);
          if (lanes < 4 || lanes > 64 || held < dim) ++bad;
        }
  for (const auto& [kind, lanes] : most) {
    const auto [inter, whole, size] = kind;
    if (lanes != head_most_lanes(inter, whole, size)) {
      std::fprintf(stderr, "interleaved %d whole %d size %d: %d lanes\n", inter, whole, size, lanes);
      ++bad;
    }
  }
  if (!bad) std::puts("ALL OK");
  return bad ? 1 : 0;
}
