// tq_attn_work.cuh -- how the kernel for many rows deals its work to thread
// blocks: integer arithmetic on q_start and kv_len alone, which the host
// compiles too.
//
// The work, every key tile of every row tile of every head, is laid in one
// line (head, sequence, row tile, key tile) and cut into equal pieces, one for
// each block: lengths, causality and the number of SMs then leave no SM idle,
// and a row tile is cut at most where a piece ends. With four blocks or more to
// a row tile, where starting and ending a second one would weigh, each row
// tile gets blocks of its own instead, as many as its share of the work.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define TQ_HD __host__ __device__ __forceinline__
#define TQ_HD_NOINLINE __host__ __device__ __noinline__
#else
#define TQ_HD inline
#define TQ_HD_NOINLINE inline
#endif

namespace tq {
namespace work {

constexpr int kHalf = 128;            // rows of a softmax
constexpr int kRows = 2 * kHalf;      // rows of a tile
constexpr int kKeys = 128;            // keys of a tile
// The cost of work, in units of about 0.4 us: a key tile of two halves, one of
// up to 128 rows, starting and ending a row tile (1.6, 1.2 and about 7 us
// measured at heads of 128, and taken for all), and the least work worth a block
// of its own.
constexpr int kCostTwo = 4, kCostAlt = 3, kTileCost = 18, kLeastWork = 12;

TQ_HD int least(int a, int b) { return a < b ? a : b; }
TQ_HD int most(int a, int b) { return a > b ? a : b; }
TQ_HD int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }
TQ_HD int64_t most(int64_t a, int64_t b) { return a > b ? a : b; }

// a / b for non-negative values: the 64-bit division, some hundred dependent
// instructions, only where it is needed.
TQ_HD_NOINLINE int64_t quotient64(int64_t a, int64_t b) { return a / b; }
TQ_HD int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : quotient64(a, b);
}

// A block's share of one row tile.
struct Segment {
  int n;              // key tiles; -1: no more segments
  int t0;             // first key tile
  int tok;            // token of the tile's first row
  int off;            // query head of that row within the group
  int rows;
  int pos;            // position of that token
  int lo, hi;         // keys [lo, hi) are seen by some row
  int head, seq;
  int part;           // where the partial result goes, -1: whole, to the output
};

// The row tiles of sequence b are numbered from f(b) = floor(q_start[b] * group
// / kRows) + b, which leaves each sequence room for all of its own (and some
// numbers empty). P has group, nseq, ntok, window (0: none) and max_positions.
template <typename P> struct Tiles {
  const P& p;
  const int32_t* q_start;   // of the call, or their copies in shared memory
  const int32_t* kv_len;
  TQ_HD int start(int b) const { return least(most(q_start[b], 0), (int)p.ntok); }
  // Whether sequence b's tokens lie within the call's, in order. A batch where
  // one's do not gets no work: the sums below search for a row tile's sequence
  // where the walk steps through them, which agree in order only.
  TQ_HD bool in_order(int b) const {
    return q_start[b] >= 0 && q_start[b] <= q_start[b + 1] && q_start[b + 1] <= p.ntok;
  }
  TQ_HD int first(int b) const { return start(b) * p.group / kRows + b; }
  // the sequence that tile number s belongs to
  TQ_HD int find(int s) const {
    int lo = 0, hi = p.nseq;   // f(lo) <= s < f(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first(mid) <= s) lo = mid;
      else hi = mid;
    }
    return lo;
  }
};

// Row tile `s` of sequence `b`, whole; n = -1 if the number is an empty one.
template <typename P> TQ_HD Segment row_tile(const Tiles<P>& tiles, int s, int b) {
  const P& p = tiles.p;
  Segment g = {};
  g.n = -1;
  const int q0 = tiles.start(b), qn = most(tiles.start(b + 1) - q0, 0);
  const int row0 = (s - tiles.first(b)) * kRows;
  if (row0 < 0 || row0 >= qn * p.group) return g;   // (below 0: q_start not in order)
  const int kv = least(most(tiles.kv_len[b], 0), p.max_positions);
  const int t = row0 / p.group;
  g.seq = b;
  g.off = row0 - t * p.group;
  g.rows = least(kRows, qn * p.group - row0);
  g.tok = q0 + t;
  g.pos = kv - qn + t;
  g.hi = most(g.pos + (g.off + g.rows - 1) / p.group + 1, 0);
  g.lo = p.window > 0 ? most(0, g.pos - p.window + 1) : 0;
  g.t0 = g.lo / kKeys;
  g.n = most((g.hi + kKeys - 1) / kKeys - g.t0, 0);
  return g;
}
TQ_HD int unit_cost(const Segment& g) { return g.rows > kHalf ? kCostTwo : kCostAlt; }
// (a tile without keys still has its rows to write)
TQ_HD int tile_cost(const Segment& g, int tile) {
  return g.n < 0 ? 0 : tile + most(g.n * unit_cost(g), 1);
}

// Some consecutive row tiles of a head: their cost, with their number above it,
// and that of starting and ending them added later. 2^19 row tiles of up to
// 2^23 key tiles fill the 63 bits; where there can be more, that cost is in the
// sum instead of the number, which only decides about blocks of their own.
constexpr int kCount = 44;
constexpr int kCounted = 1 << 19;     // row tile numbers, of which so many are counted
template <typename P> TQ_HD int64_t sum_tiles(const Tiles<P>& tiles, int numbers, int i0, int i1, int b0) {
  const int64_t each = numbers < kCounted ? int64_t(1) << kCount : kTileCost;
  int64_t sum = 0;
  for (int s = i0, b = b0; s < i1; ++s) {
    while (b + 1 < tiles.p.nseq && tiles.first(b + 1) <= s) ++b;
    const int cost = tile_cost(row_tile(tiles, s, b), 0);
    sum += cost > 0 ? cost + each : 0;
  }
  return sum;
}

// Where a block's work starts: a row tile's number and sequence, its head, and
// the cost before it.
struct Start {
  int number, seq, head, own;
  int64_t x0, x1;     // the block's piece of the line (own: x0 row tiles before)
  int64_t at;
  int64_t all, blocks, spare;
};

// Whether the work of `block` of `grid` starts in the row tiles [i0, ..) with
// the sum `mine` (the first of them in sequence b0), `before` those before
// them and `total` all of a head; and where.
TQ_HD bool find_start(int64_t before, int64_t mine, int64_t total, int numbers, int i0, int b0, int heads,
                      int64_t block, int64_t grid, Start* start) {
  const bool counted = numbers < kCounted;
  const bool own = total == 0 || (counted && (total >> kCount) * heads * 4 <= grid);
  const int tile_fee = own ? 0 : kTileCost;
  auto cost_of = [&](int64_t sum) {
    return counted ? (sum & ((int64_t(1) << kCount) - 1)) + (sum >> kCount) * tile_fee : sum;
  };
  const int64_t tiles_before = before >> kCount, tiles_mine = mine >> kCount;
  const int64_t head_tiles = total >> kCount;
  total = cost_of(total);
  before = cost_of(before);
  mine = cost_of(mine);
  const int64_t all = total * heads;
  // as many blocks as there is work for
  const int64_t blocks = most((int64_t)1, least(grid, quotient(all, kLeastWork)));
  // own: every row tile has blocks of its own, those of the tile number i that
  // has the cost `sum` before it from first_block(i, sum) on
  const int64_t spare = own ? most(blocks - head_tiles * heads, (int64_t)0) : 0;
  auto first_block = [&](int64_t i, int64_t sum) { return i + quotient(sum * spare, most(all, (int64_t)1)); };
  int64_t x0 = all, x1 = all;   // !own: the block's piece of the line
  int head0 = 0;                // the head its first row tile belongs to
  bool here;
  if (own) {
    while (head0 + 1 < heads && first_block((head0 + 1) * head_tiles, (head0 + 1) * total) <= block) ++head0;
    const int64_t i = head0 * head_tiles + tiles_before, sum = head0 * total + before;
    here = mine > 0 && first_block(i, sum) <= block && block < first_block(i + tiles_mine, sum + mine);
    x0 = i;
    x1 = sum;
  } else {
    if (block < blocks) {
      x0 = quotient(all * block, blocks);
      x1 = quotient(all * (block + 1), blocks);
      head0 = (int)quotient(x0, total);
    }
    const int64_t y0 = x0 - head0 * total;
    here = block < blocks && mine > 0 && before <= y0 && y0 < before + mine;
  }
  if (here) *start = {i0, b0, head0, own, x0, x1, own ? x1 : head0 * total + before, all, blocks, spare};
  return here;
}

// A row tile that was cut: its rows, and where its partial results are.
struct CutTile {
  int n;              // pieces; 0: none here
  int part0;          // the first, then 2 (block + 1), 2 (block + 2), ...
  int tok, off, rows, head;
  int pad[2];
};

// The block's work from `st` on: push(segment) for each of its row tiles, in
// order, until stop(); the row tile that was cut and whose first piece is here.
// Whatever q_start holds, heads and pieces stay within `heads` and `grid`.
template <typename P, typename Push, typename Stop>
TQ_HD CutTile walk(const Tiles<P>& tiles, int numbers, const Start& st, int heads, int grid, int block,
                   Push push, Stop stop) {
  CutTile cut = {};
  int pushed = 0;
  int s = st.number, b = st.seq;   // number of the row tile, its sequence
  if (s < 0) return cut;
  if (st.own) {
    int64_t i = st.x0, sum = st.at;
    for (; s < numbers; ++s) {
      while (b + 1 < tiles.p.nseq && tiles.first(b + 1) <= s) ++b;
      Segment g = row_tile(tiles, s, b);
      const int cost = tile_cost(g, 0);
      if (cost == 0) continue;
      const int64_t from = i + quotient(sum * st.spare, st.all);
      const int64_t to = i + 1 + quotient((sum + cost) * st.spare, st.all);
      ++i;
      sum += cost;
      if ((int64_t)block >= to) continue;
      // piece j of `pieces` (none without a key tile, but for the only one)
      const int j = (int)(block - from), n = g.n;
      const int pieces = most(least((int)(to - from), n), 1);
      if (j < pieces) {
        const int t0 = (int)quotient((int64_t)n * j, pieces), t1 = (int)quotient((int64_t)n * (j + 1), pieces);
        g.head = st.head;
        g.part = pieces == 1 ? -1 : 2 * block;
        if (pieces > 1 && j == 0) cut = {pieces, g.part, g.tok, g.off, g.rows, g.head, {}};
        g.t0 += t0;
        g.n = t1 - t0;
        push(g);
      }
      break;
    }
    return cut;
  }
  int head = st.head;
  int64_t at = st.at;   // start of the row tile
  while (at < st.x1 && head < heads && !stop()) {
    while (b + 1 < tiles.p.nseq && tiles.first(b + 1) <= s) ++b;
    Segment g = row_tile(tiles, s, b);
    const int cost = tile_cost(g, kTileCost);
    if (cost > 0 && at + cost > st.x0) {
      // key tiles [from, to) of the row tile fall into the piece
      const int w = unit_cost(g), n = g.n;
      const int u0 = (int)most(st.x0 - at, (int64_t)0), u1 = (int)least(st.x1 - at, (int64_t)cost);
      const int from = u0 < kTileCost ? 0 : least((u0 - kTileCost) / w, n);
      const int to = u1 < kTileCost ? 0 : least((u1 - kTileCost) / w, n);
      if (n == 0 ? u0 == 0 : from < to) {
        g.head = head;
        g.part = from == 0 && to == n ? -1 : 2 * block + (pushed > 0);
        if (g.part >= 0 && from == 0) {
          // up to the piece with the row tile's end
          const int64_t last = quotient((at + cost) * st.blocks + st.all - 1, st.all) - 1;
          cut = {least((int)(last - block) + 1, grid - block), g.part, g.tok, g.off, g.rows, g.head, {}};
        }
        g.t0 += from;
        g.n = to - from;
        push(g);
        ++pushed;
      }
    }
    at += cost;
    if (++s == numbers) {
      s = 0;
      b = 0;
      ++head;
    }
  }
  return cut;
}

}  // namespace work
}  // namespace tq
