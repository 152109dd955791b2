// The shared-prefix attention's work on the host: which blocks its warps and CTAs leave, one of them giving up on the way,
// and which its join reads (td_runs.cuh). Return 0, or the line of the first rule that does not hold.
#include <algorithm>
#include <vector>

#include "td_runs.cuh"

#define HOLDS(x) \
  if (!(x)) return __LINE__

namespace {
constexpr int D = 64;
enum : int { kBefore = 7, kKeys = 1, kNone = 0 };  // a block's sums l: an earlier call's, this call's, without keys
}  // namespace

// The runs of `grid` CTAs over B sequences of len[b] keys, Hkv * RB groups of R rows each. Run `quits` gives up in its
// `after`-th group (from 0). *met: the groups behind it that it leaves.
extern "C" int check_runs(int B, int Hkv, int RB, int R, int grid, const int *len, int quits, int after, int *met) {
  const int U = Hkv * RB, runs = grid * td::kRunWarps, BF = td::run_block_floats(R, D);
  std::vector<int> prefix(B + 1, 0);
  for (int b = 0; b < B; ++b) prefix[b + 1] = prefix[b] + td::run_units(len[b]) * U;
  const int S = td::run_length(prefix[B], grid);
  std::vector<float> ws((size_t)(B * U + runs) * BF, kBefore);
  td::SplitParams p = {};
  p.B = B, p.Hkv = Hkv, p.RB = RB, p.R = R, p.ws_part = ws.data();
  auto sums = [&](int g, int r) { return ws.data() + td::run_block(g, r) * BF + R * (D + 1); };
  int steps = 0;
  *met = 0;
  for (int r = 0; r < runs; ++r) {
    int u1;
    td::RunCursor c = td::run_start(p, len, prefix.data(), S, r, u1);
    for (int n = 0; c.s < c.e; ++n) {
      const int g = c.b * U + c.ug;
      HOLDS(c.b < B && c.ug < U && c.e <= td::run_steps(len[c.b]));
      HOLDS(sums(g, r)[0] == kBefore);  // a block of its own
      steps += c.e - c.s;
      const bool quit = r == quits && n == after;
      std::fill_n(sums(g, r), R, float(quit ? kNone : kKeys));
      if (quit) {
        td::RunCursor left = c;
        for (td::next_group(p, len, u1, left); left.s < left.e; td::next_group(p, len, u1, left)) {
          steps += left.e - left.s;
          ++*met;
        }
        for (int lane = 0; lane < 32; ++lane) td::drop_rest_of_run<D>(p, len, c, u1, r, lane, 32);
        break;
      }
      td::next_group(p, len, u1, c);
    }
  }
  int all = 0, blocks = 0;
  for (int b = 0; b < B; ++b)
    for (int ug = 0; ug < U; ++ug) {
      const int units = td::run_units(len[b]);
      const td::RunSpan span = td::runs_of(prefix[b] + ug * units, units, S);
      all += units > 0 ? td::run_steps(len[b]) : 0;
      HOLDS((span.n > 0) == (len[b] > 0));
      for (int r = span.first; r < span.first + span.n; ++r, ++blocks)
        for (int i = 0; i < R; ++i) HOLDS(sums(b * U + ug, r)[i] == kKeys || (r == quits && sums(b * U + ug, r)[i] == kNone));
    }
  HOLDS(steps == all);  // every step is some run's, once
  int left = 0;
  for (int i = 0; i < B * U + runs; ++i) left += ws[(size_t)i * BF + R * (D + 1)] != kBefore;
  HOLDS(left == blocks);
  return 0;
}

// The tiles of `tiles` x 128 rows of Hkv kv heads over a prefix of P keys cut into at most `chunks`. CTA `quits` gives up.
extern "C" int check_items(int tiles, int Hkv, int chunks, int grid, int P, int quits) {
  constexpr int BF = td::prefix_block_floats(D), L = td::kPrefixRows * (D + 1);
  std::vector<float> part((size_t)tiles * Hkv * chunks * BF, kBefore);
  auto sums = [&](int kvh, int tile, int c) { return part.data() + td::prefix_block(kvh, tile, c, tiles, chunks) * BF + L; };
  const int C = td::prefix_chunk(P, chunks);
  for (int cta = 0; cta < grid; ++cta) {
    for (int item = cta; item < (P > 0 ? tiles * Hkv * chunks : 0); item += grid) {
      const td::PrefixItem w = td::prefix_item(item, tiles, Hkv);
      if (std::min(w.chunk * C, P) == P) break;  // later items are of the same or a later chunk
      HOLDS(sums(w.kvh, w.tile, w.chunk)[0] == kBefore);
      std::fill_n(sums(w.kvh, w.tile, w.chunk), td::kPrefixRows, float(kKeys));
    }
    if (cta == quits)
      for (int lane = 0; lane < td::kPrefixRows; ++lane)
        td::drop_items<D>(part.data(), P, tiles, Hkv, chunks, cta, grid, lane, td::kPrefixRows);
  }
  int none = 0;
  for (int kvh = 0; kvh < Hkv; ++kvh)
    for (int tile = 0; tile < tiles; ++tile)
      for (int c = 0; c < chunks; ++c)
        for (int i = 0; i < td::kPrefixRows; ++i) {
          const float l = sums(kvh, tile, c)[i];
          HOLDS(c < td::prefix_parts(P, chunks) ? l == kKeys || l == kNone : l == kBefore);
          none += l == kNone;
        }
  int its = 0;
  for (int item = quits; item < tiles * Hkv * td::prefix_parts(P, chunks); item += grid) ++its;
  HOLDS(none == its * td::kPrefixRows);
  return 0;
}
