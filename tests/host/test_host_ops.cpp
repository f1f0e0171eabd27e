// Host-only checks of the training operators' argument validation, built with
// g++ and AddressSanitizer / UndefinedBehaviorSanitizer by
// tests/test_host_ops.py (validate_ops.cpp makes no HIP call).  Prints
// "ALL OK" and exits 0 when every check holds.
#include <cmath>
#include <cstdio>
#include <limits>
#include <string>

#include "../../newton_schulz_05_amd/csrc/validate_ops.hpp"

using namespace muon;

static int g_fail = 0;
#define CHECK(cond)                                                                 \
  do {                                                                              \
    if (!(cond)) {                                                                  \
      std::fprintf(stderr, "%s:%d: CHECK failed: %s\n", __FILE__, __LINE__, #cond); \
      ++g_fail;                                                                     \
    }                                                                               \
  } while (0)

static Operand op(uint64_t at, int64_t rows, int64_t width, int64_t pitch, bool written = false) {
  return {"t", reinterpret_cast<const void*>(uintptr_t(at)), rows, width, pitch, 1, written, false};
}

// overlap() against the bytes themselves, over every small layout.
static void check_overlap() {
  for (int64_t ra = 1; ra <= 3; ++ra)
    for (int64_t rb = 1; rb <= 3; ++rb)
      for (int64_t wa = 1; wa <= 4; ++wa)
        for (int64_t wb = 1; wb <= 4; ++wb)
          for (int64_t pitch = 4; pitch <= 7; ++pitch)
            for (int64_t d = -22; d <= 22; ++d) {
              const Operand a = op(1000, ra, wa, pitch), b = op(uint64_t(1000 + d), rb, wb, pitch);
              bool share = false;
              for (int64_t i = 0; i < ra; ++i)
                for (int64_t j = 0; j < rb; ++j) {
                  const int64_t x = i * pitch, y = d + j * pitch;
                  share = share || (x < y + wb && y < x + wa);
                }
              if (share) CHECK(overlap(a, b));
              // never refused: runs that lie apart within the pitch, or ranges that do not meet
              const int64_t m = ((d % pitch) + pitch) % pitch;
              if (m >= wa && m + wb <= pitch) CHECK(!overlap(a, b) || (ra == 1 && rb == 1 && share));
              CHECK(overlap(a, b) == overlap(b, a));
            }
}

int main() {
  check_overlap();
  std::string d;
  const int64_t top = std::numeric_limits<int64_t>::max(), low = std::numeric_limits<int64_t>::min();
  CHECK(check_rows(0, 1, 8, {1}, &d) == MUON_OK);
  CHECK(check_rows(top, 1, 8, {1}, &d) == MUON_ERR_SHAPE);
  CHECK(check_rows(low, 1, 8, {1}, &d) == MUON_ERR_SHAPE);
  CHECK(check_rows(1, low, 8, {1}, &d) == MUON_ERR_SHAPE);
  CHECK(check_rows(1, 4, 8, {top}, &d) == MUON_ERR_SHAPE);
  CHECK(check_rows(1, 4, 8, {low}, &d) == MUON_ERR_INVALID_ARG);
  CHECK(check_rows(int64_t(1) << 40, 4, 8, {int64_t(1) << 40}, &d) == MUON_ERR_SHAPE);
  CHECK(check_rows(1, 4, 8, {int64_t(1) << 40}, &d) == MUON_OK);
  CHECK(check_dropout(std::nanf(""), 1, nullptr, &d) == MUON_ERR_INVALID_ARG);
  CHECK(check_dropout(0.5f, int64_t(1) << 32, nullptr, &d) == MUON_ERR_SHAPE);
  CHECK(check_dropout(1.0f, (int64_t(1) << 32) - 1, nullptr, &d) == MUON_OK);
  CHECK(check_route(top, 8, 8, 1, 0, 1.0f, MUON_F32, &d) == MUON_ERR_SHAPE);
  CHECK(check_route(0x7fffffff, 8, 8, 1, 0, 1.0f, MUON_F32, &d) == MUON_OK);
  CHECK(check_route(0x7fffffff, 8, 8, 2, 0, 1.0f, MUON_F32, &d) == MUON_ERR_SHAPE);
  // the workspace of every width is a whole number of partial sums, and stays
  // below a bound that holds for any number of rows
  for (int64_t cols = 1; cols <= kNormMaxCols; cols = cols * 3 / 2 + 1)
    for (int64_t rows : {int64_t(0), int64_t(1), int64_t(511), int64_t(70000), int64_t(1) << 40}) {
      const NormBwdSplit sp = norm_bwd_split(rows, cols);
      CHECK(sp.parts >= 0 && sp.parts <= kNormMaxParts && (sp.parts == 0) == (rows <= kNormFewRows));
      CHECK(sp.threads % sp.row_threads == 0 && sp.threads >= 256 && sp.threads <= 1024);
      CHECK(norm_workspace_bytes(rows, cols) == size_t(sp.parts) * 2 * cols * 4);
    }
  for (int64_t e = 1; e <= kRouteMaxExperts; ++e) {
    CHECK(route_workspace_bytes(0, e) == 0 && route_workspace_bytes(1000, e) > 0);
    CHECK((e + 15) / 16 <= kRouteTerms && route_parts(int64_t(1) << 31, e) <= kRouteMaxParts);
    CHECK(route_parts(1, e) == 1 && route_parts(int64_t(1) << 31, e) >= 1);
  }
  if (g_fail) return 1;
  std::puts("ALL OK");
  return 0;
}
