// Host-only checks of the argument validation and work splits of the operators
// at the two ends of a training step, built with g++ and AddressSanitizer /
// UndefinedBehaviorSanitizer by tests/test_host_ends.py.  Prints "ALL OK" and
// exits 0 when every check holds.
#include <cmath>
#include <cstdio>
#include <limits>
#include <set>
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

// Bytes of a tensor of heads; false if an element comes twice.
static bool bytes(int64_t b, int64_t t, int64_t h, int64_t dim, const muon_head_strides& s, std::set<int64_t>* out) {
  for (int64_t i = 0; i < b; ++i)
    for (int64_t j = 0; j < t; ++j)
      for (int64_t k = 0; k < h; ++k)
        for (int64_t e = 0; e < dim; ++e)
          if (!out->insert(i * s.batch + j * s.token + k * s.head + e).second) return false;
  return true;
}

// Over every small set of strides: an accepted tensor names no element twice, its
// runs cover its bytes and begin with it, and column slices of one buffer are apart.
static void check_head_operands() {
  std::string d;
  int accepted = 0;
  for (int64_t b = 1; b <= 2; ++b)
    for (int64_t t = 1; t <= 3; ++t)
      for (int64_t h = 1; h <= 2; ++h)
        for (int64_t sb = 0; sb <= 14; ++sb)
          for (int64_t st = 0; st <= 14; ++st)
            for (int64_t sh = 0; sh <= 14; ++sh) {
              const muon_head_strides s{sb, st, sh};
              Operand o;
              if (head_operand("t", reinterpret_cast<void*>(0x1000), &s, b, t, h, 2, 1, false, &o, &d) != MUON_OK) continue;
              ++accepted;
              std::set<int64_t> own;
              CHECK(bytes(b, t, h, 2, s, &own));
              CHECK(*own.begin() == 0 && o.rows >= 1 && o.width >= 2 && (o.rows == 1 || o.width <= o.pitch));
              CHECK((o.rows - 1) * o.pitch + o.width == *own.rbegin() + 1);
              for (int64_t e : own) CHECK(e / o.pitch < o.rows && e % o.pitch < o.width);
            }
  CHECK(accepted > 1000);
  // slices of a projection's output: 3 tokens of (2 + 1 + 1) heads of 4
  const muon_head_strides s{48, 16, 4};
  Operand q, k, v;
  CHECK(head_operand("q", reinterpret_cast<void*>(0x1000), &s, 2, 3, 2, 4, 1, true, &q, &d) == MUON_OK);
  CHECK(head_operand("k", reinterpret_cast<void*>(0x1008), &s, 2, 3, 1, 4, 1, true, &k, &d) == MUON_OK);
  CHECK(head_operand("v", reinterpret_cast<void*>(0x1006), &s, 2, 3, 1, 4, 1, true, &v, &d) == MUON_OK);
  CHECK(!overlap(q, k) && overlap(q, v) && overlap(k, v));
  const int64_t top = std::numeric_limits<int64_t>::max(), low = std::numeric_limits<int64_t>::min();
  for (int64_t x : {top, low, int64_t(1) << 41, int64_t(-1)}) {
    const muon_head_strides w{x, 16, 4};
    CHECK(head_operand("w", reinterpret_cast<void*>(0x1000), &w, 2, 3, 2, 4, 2, true, &q, &d) != MUON_OK);
    CHECK(head_operand("w", reinterpret_cast<void*>(0x1000), &w, 1, 3, 2, 4, 2, true, &q, &d) == MUON_OK);
  }
}

// Overlap of two tensors of heads with common strides, against their bytes: slices
// of tokens and of heads of one buffer, every distance.
static void check_head_overlap() {
  std::string d;
  int apart = 0, met = 0;
  for (int64_t st : {8, 9, 12})
    for (int64_t sb : {2 * st, 3 * st, 3 * st + 5})
      for (int64_t sh : {2, 3})
        for (int64_t t = 1; t <= 2; ++t)
          for (int64_t ha = 1; ha <= 2; ++ha)
            for (int64_t hb = 1; hb <= 2; ++hb)
              for (int64_t at = -40; at <= 40; ++at) {
                const muon_head_strides s{sb, st, sh};
                Operand a, b;
                CHECK(head_operand("a", reinterpret_cast<void*>(0x1000), &s, 2, t, ha, 2, 1, true, &a, &d) == MUON_OK);
                CHECK(head_operand("b", reinterpret_cast<void*>(uintptr_t(0x1000 + at)), &s, 2, t, hb, 2, 1, true, &b, &d) == MUON_OK);
                std::set<int64_t> x, y;
                bytes(2, t, ha, 2, s, &x);
                bytes(2, t, hb, 2, s, &y);
                bool share = false;
                for (int64_t e : y) share = share || x.count(e + at);
                CHECK(overlap(a, b) == share && overlap(b, a) == share);
                ++(share ? met : apart);
              }
  CHECK(apart > 1000 && met > 1000);
}

static void check_fast_div() {
  for (int64_t d = 2; d < 0x7fffffff; d = d < 3000 ? d + 1 : d * 5 / 4 + 1) {
    const FastDiv f = fast_div(d);
    auto q = [&](uint64_t r) { return int64_t(((r * f.mul) >> 32) >> f.shift); };
    for (int64_t r : {int64_t(0), d - 1, d, d + 1, 2 * d - 1, 2 * d, int64_t(0x7ffffffe), int64_t(0x7fffffff),
                      0x7fffffff / d * d, 0x7fffffff / d * d - 1, 0x40000000 / d * d, 0x40000000 / d * d - 1})
      if (r >= 0 && r <= 0x7fffffff) CHECK(q(uint64_t(r)) == r / d);
  }
}

int main() {
  check_head_operands();
  check_head_overlap();
  check_fast_div();
  std::string d;
  const int64_t top = std::numeric_limits<int64_t>::max();
  auto heads = [&](int64_t b, int64_t t, int32_t hq, int32_t hk, int64_t table, int64_t posb) {
    const float f = 0;
    const int64_t p = 0;
    return check_heads(MUON_F32, MUON_F32, b, t, hq, hk, hk != 0, 8, 1e-6f, &f, &f, table, 8, 0, &p, posb, &d);
  };
  CHECK(heads(1, 1, 1, 0, 1, 0) == MUON_OK && heads(1, 0x7fffffff, 1, 1, 1, 0) == MUON_OK);
  CHECK(heads(2, 0x7fffffff, 1, 1, 1, 0) == MUON_ERR_SHAPE);
  CHECK(heads(top, top, 1, 1, 1, 0) == MUON_ERR_SHAPE && heads(1, 1, 0x7fffffff, 1, 1, 0) == MUON_OK);
  CHECK(heads(1, 2, 0x7fffffff, 1, 1, 0) == MUON_ERR_SHAPE && heads(1, 1, 1, 0x7fffffff, 1, 0) == MUON_OK);
  CHECK(heads(2, 4, 1, 1, top, 4) == MUON_ERR_SHAPE && heads(2, 4, 1, 1, 5, top) == MUON_ERR_SHAPE);
  CHECK(check_logp(0x7fffffff, 1 << 24, {int64_t(1) << 24}, MUON_BF16, 1.0f, &d) == MUON_ERR_SHAPE);
  CHECK(check_logp(1000, 1 << 24, {int64_t(1) << 24}, MUON_BF16, 1.0f, &d) == MUON_OK);
  CHECK(check_logp(1, 4, {top}, MUON_F32, 1.0f, &d) == MUON_ERR_SHAPE);
  CHECK(check_policy(top, 0, 0, 0, &d) == MUON_ERR_SHAPE && check_preference(top, 0, 0, 0, 0, 0, &d) == MUON_ERR_SHAPE);

  // lanes cover every element of a row
  for (int dim = 1; dim <= kHeadMaxDim; ++dim)
    for (int rot = 0; rot <= dim; rot += 2)
      for (bool inter : {false, true}) {
        const int lanes = head_lanes(dim, rot, inter), first = inter ? 0 : (rot / 2 + 7) / 8;
        CHECK(lanes <= 64 && (inter ? 16 * lanes >= dim : first <= lanes && 16 * (lanes - first) >= dim - rot));
      }
  // splits: within their bounds for any number of rows, and never without a workgroup
  for (int64_t q : {int64_t(1), int64_t(63), int64_t(64), int64_t(65), int64_t(70000), kHeadMaxRows})
    for (int64_t k : {int64_t(0), int64_t(1), int64_t(64), int64_t(9000), kHeadMaxRows}) {
      const HeadSplit s = head_split(q, k);
      CHECK(s.q >= 1 && (k > 0 ? s.k >= 1 : s.k == 0) && s.q + s.k <= kHeadMaxParts + 1);
      CHECK(heads_workspace_bytes(q, k, 512) <= size_t(kHeadMaxParts + 1) * 2048);
    }
  CHECK(head_split(0, 0).q == 0 && head_split(0, 0).k == 0 && heads_workspace_bytes(0, 0, 8) == 0);
  for (int64_t rows : {int64_t(0), int64_t(1), int64_t(2), int64_t(511), int64_t(512), kHeadMaxRows})
    for (int64_t vocab = 1; vocab <= kLogpMaxVocab; vocab = vocab * 2 + 1) {
      const int parts = logp_parts(rows, vocab);
      CHECK(parts >= 1 && parts <= kLogpMaxParts && (rows < 512 || parts == 1));
    }
  for (int64_t n : {int64_t(0), int64_t(1), int64_t(4096), int64_t(4097), kLossMaxTokens}) {
    CHECK(policy_parts(n) >= 1 && policy_parts(n) <= kPolicyMaxParts);
    for (int64_t p : {int64_t(0), int64_t(1), kPrefMaxPairs})
      CHECK(pref_shift(n, p) >= 0 && (1 << pref_shift(n, p)) <= kPrefMaxChunks);
  }
  if (g_fail) return 1;
  std::puts("ALL OK");
  return 0;
}
