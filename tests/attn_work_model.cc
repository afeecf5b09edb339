// The blocks of the many-row attention kernel as a host program: every thread's sum, the scan, the
// start and the walk, on the kernel's own arithmetic, and what the blocks then do with the segments.
#include <cstdio>
#include <cstring>
#include <vector>

#include "../bit_matvec_gb300/csrc/tq_attn_work.cuh"

using namespace tq::work;

namespace {
struct Params {
  int group, nseq;
  int64_t ntok;
  int window, max_positions;
};
constexpr int kThreads = 384;

struct Piece {
  Segment g;
  int block;
};
bool fails(char* why, const char* what, long long a = 0, long long b = 0) {
  if (why[0] == 0) snprintf(why, 256, "%s (%lld, %lld)", what, a, b);
  return false;
}
}  // namespace

// Whether all of it stays in bounds, and, for a `sound` batch, every row tile of every head is covered
// once, by one whole segment or by pieces that the join finds. `why` (256 bytes) says what is wrong.
extern "C" int attn_work_check(const int32_t* q_start, const int32_t* kv_len, int nseq, int64_t ntok,
                               int group, int heads, int window, int max_positions, int grid, int sound,
                               char* why) {
  why[0] = 0;
  const Params p{group, nseq, ntok, window, max_positions};
  const Tiles<Params> tiles{p, q_start, kv_len};
  const int numbers = (int)(ntok * group / kRows + nseq);
  const int per = (numbers + kThreads - 1) / kThreads;
  struct Mine {
    int i0, b0;
    int64_t before, mine;
  };
  std::vector<Mine> threads(kThreads);
  int64_t total = 0;
  for (int t = 0; t < kThreads; ++t) {
    const int i0 = least(t * per, numbers), i1 = least(i0 + per, numbers);
    const int b0 = i0 < i1 ? tiles.find(i0) : 0;
    const int64_t mine = sum_tiles(tiles, numbers, i0, i1, b0);
    threads[t] = {i0, b0, total, mine};
    total = total + mine;
  }
  std::vector<Piece> pieces;
  std::vector<CutTile> cuts(grid);
  for (int block = 0; block < grid; ++block) {
    Start st = {};
    st.number = -1;
    int starts = 0;
    for (const Mine& m : threads)
      starts += find_start(m.before, m.mine, total, numbers, m.i0, m.b0, heads, block, grid, &st);
    if (starts > 1) return fails(why, "several starts of block", block, starts);
    int steps = 0;
    const size_t first = pieces.size();
    cuts[block] = walk(tiles, numbers, st, heads, grid, block,
                       [&](const Segment& g) { pieces.push_back({g, block}); },
                       [&]() { return ++steps > 100000000; });
    if (steps > 100000000) return fails(why, "no end of the walk of block", block);
    // a block has room for two partial results: its first row tile's and its last's
    int parts[2] = {0, 0};
    for (size_t i = first; i < pieces.size(); ++i) {
      const Segment& g = pieces[i].g;
      if (g.head < 0 || g.head >= heads) return fails(why, "head of block", g.head, block);
      if (g.seq < 0 || g.seq >= nseq) return fails(why, "sequence", g.seq, block);
      if (g.rows < 1 || g.rows > kRows || g.off < 0 || g.off >= group) return fails(why, "rows", g.rows, g.off);
      if (g.tok < 0 || g.tok + (g.off + g.rows - 1) / group >= ntok) return fails(why, "token", g.tok, block);
      if (g.n < 0 || g.t0 < 0 || (int64_t)(g.t0 + g.n) * kKeys > (int64_t)max_positions + kKeys)
        return fails(why, "key tiles", g.t0, g.n);
      if (g.part >= 0) {
        if (g.part / 2 != block) return fails(why, "partial result of block", g.part, block);
        ++parts[g.part % 2];
      }
    }
    if (parts[0] > 1 || parts[1] > 1) return fails(why, "one place for two partial results", block);
  }
  // the join reads the places of a cut row tile's pieces
  for (int block = 0; block < grid; ++block)
    for (int i = 0; i < cuts[block].n; ++i) {
      const int64_t at = i == 0 ? cuts[block].part0 : 2 * (block + i);
      if (at < 0 || at >= 2 * grid) return fails(why, "join past the partial results", block, at);
    }
  if (!sound) return 1;

  // every (head, row tile): its key tiles covered in order
  std::vector<std::vector<Piece>> of((size_t)heads * numbers);
  for (const Piece& x : pieces) {
    const Segment& g = x.g;
    const int row = (int)((g.tok - tiles.start(g.seq)) * group + g.off);
    if (row % kRows) return fails(why, "first row", row);
    of[(size_t)g.head * numbers + tiles.first(g.seq) + row / kRows].push_back(x);
  }
  for (int h = 0; h < heads; ++h)
    for (int s = 0, b = 0; s < numbers; ++s) {
      while (b + 1 < nseq && tiles.first(b + 1) <= s) ++b;
      const Segment g = row_tile(tiles, s, b);
      const std::vector<Piece>& v = of[(size_t)h * numbers + s];
      if (g.n < 0) {
        if (!v.empty()) return fails(why, "work for an empty number", s);
        continue;
      }
      if (v.empty()) return fails(why, "row tile left out", h, s);
      int t = g.t0;
      for (size_t i = 0; i < v.size(); ++i) {
        const Segment& x = v[i].g;
        if (x.t0 != t || x.rows != g.rows || x.pos != g.pos || x.hi != g.hi || x.lo != g.lo)
          return fails(why, "piece of row tile", h, s);
        t += x.n;
        if ((x.part < 0) != (v.size() == 1)) return fails(why, "whole or piece", h, s);
      }
      if (t != g.t0 + g.n) return fails(why, "end of row tile", h, s);
      if (v.size() > 1) {
        const CutTile& c = cuts[v[0].block];
        if (c.n != (int)v.size() || c.tok != g.tok || c.off != g.off || c.rows != g.rows || c.head != h)
          return fails(why, "cut of row tile", h, s);
        for (size_t i = 0; i < v.size(); ++i)
          if (v[i].g.part != (i == 0 ? c.part0 : 2 * (v[0].block + (int)i)))
            return fails(why, "place of piece", h, s);
      }
    }
  int cut = 0, joined = 0;
  for (const auto& v : of) cut += v.size() > 1;
  for (const CutTile& c : cuts) joined += c.n > 0;
  return cut == joined ? 1 : fails(why, "row tiles joined", cut, joined);
}
