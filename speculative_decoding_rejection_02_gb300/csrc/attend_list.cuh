// The list of key tiles that an attention call works through (cache_attend.cuh),
// and a block's walk over its part of it: arithmetic alone, which also compiles
// as plain C++ for the tests.
//
// A unit is up to two tiles of rows of one request and kv head. It takes its key
// tiles and a fixed number of places more, which stand for what its start and its
// results cost. The list is all units in order of request, kv head and rows, and
// is never written down: a block finds its part from the requests' lengths.
#pragma once
#ifdef __CUDACC__
#define SV_LIST __device__ __forceinline__
#else
#include <algorithm>
#define SV_LIST inline
#endif

namespace sv {

#ifndef __CUDACC__
using std::max;
using std::min;
#endif

constexpr int kAttTile = 128;     // rows of a tile, and tokens of a key tile
// What a unit costs beside its key tiles, in tiles: of one tile of rows, and of two.
constexpr int kAttCost = 2, kAttPairCost = 4;

// A unit that starts in one block's part of the list and ends in another's.
struct AttJoin {
  int last;              // its last block; -1: none
  int head, token, tokens;  // rows: new tokens token .. token + tokens - 1
};

// One entry of a block's walk: key tiles i0 .. i0 + n - 1 of a unit.
struct AttSeg {
  int n;          // key tiles here; 0: the end of the walk
  int i0;         // the first one's number within the unit
  int b, head;
  int token, tokens;  // rows of q
  int pos;        // position of the first row's token
  int lo, hi;     // tokens that some row sees: [lo, hi) and [0, min(sinks, lo))
  int gap_at, gap;  // tile i of the unit is tile i, from gap_at on tile i + gap
  int pair;       // 1: two tiles of rows; 0: even and odd key tiles
  int q_at;       // Q tiles loaded before
  unsigned ring;  // K and V tiles loaded before
  int slot;       // partial result: 0 or 1; -1: the unit is whole
};

// sum over 0 <= i < n of floor((a i + b) / m); a, b >= 0, m > 0, and a n + b and the sum
// below 2^32. The sum counts the points with whole coordinates under a line. Whole multiples
// of m in a and b are counted at once; what is left is counted along the other axis, where a
// and m have changed places: the steps of Euclid's algorithm for a and m.
SV_LIST unsigned floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  unsigned sum = 0;
  while (n > 0) {
    if (a >= m) {
      sum += (unsigned)((unsigned long long)(n - 1) * n / 2) * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += n * (b / m);
      b %= m;
    }
    const unsigned y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const unsigned t = m;
    m = a;
    a = t;
  }
  return sum;
}

// The units of one request: `count` of `step` new tokens each (the last may
// have fewer), for each kv head. Positions, and the key tiles of one head's
// units together, are below 2^31.
struct AttUnits {
  int p0;  // position of the first new token
  int q, step, count, window, sink_tiles, cost;

  SV_LIST AttUnits(int len, int q_, int step_, int window_, int sinks)
      : p0(len - q_), q(q_), step(step_), count(q_ <= step_ ? q_ > 0 : (q_ - 1) / step_ + 1),
        window(window_), sink_tiles((int)(((unsigned)sinks + kAttTile - 1) / kAttTile)),
        cost(q_ > step_ / 2 ? kAttPairCost : kAttCost) {}

  SV_LIST int hi(int u) const {
    const int end = (u + 1) * step;
    return p0 + (u + 1 < count && end < q ? end : q);
  }
  SV_LIST int lo(int u) const {
    const int first = p0 + u * step + 1;
    return window && first > window ? first - window : 0;
  }
  SV_LIST int gap(int u) const {
    const int g = lo(u) / kAttTile - sink_tiles;
    return g > 0 ? g : 0;
  }
  // Key tiles of unit u; one (in which no row sees anything) at least.
  SV_LIST int tiles(int u) const {
    const int h = hi(u);
    return h <= 0 ? 1 : (h - 1) / kAttTile + 1 - gap(u);
  }
  // Length in the list of the units before k, in closed form.
  SV_LIST int before(int k) const {
    int sum = k * cost;
    if (k == count && k > 0) sum += tiles(--k);  // the last one ends where the request does
    if (k <= 0) return sum;
    int dead = p0 < 0 ? -p0 / step : 0;  // units before position 0
    if (dead > k) dead = k;
    if (dead < k)
      sum += floor_sum(k - dead, kAttTile, step, p0 + (dead + 1) * step + kAttTile - 1);
    sum += dead;
    if (window) {
      const long long from =
          (long long)(sink_tiles + 1) * kAttTile + window - 1 - p0;  // gap > 0
      const long long u = from > 0 ? (from + step - 1) / step : 0;
      if (u < k)
        sum -= (int)floor_sum(k - (int)u, kAttTile, step, (unsigned)(p0 + u * step - window + 1)) -
               (k - (int)u) * sink_tiles;
    }
    return sum;
  }
};

// The list's part of block c begins at tile att_begin(c): the first total % blocks parts are
// a tile longer.
SV_LIST int att_begin(int c, int total, int blocks) {
  return c * (total / blocks) + min(c, total % blocks);
}
SV_LIST int att_block_of(int tile, int total, int blocks) {
  const int part = total / blocks, more = total % blocks;
  return tile < more * (part + 1) ? tile / (part + 1) : more + (tile - more * (part + 1)) / part;
}

// Number of the entry's key tile i.
SV_LIST int att_tile(const AttSeg& g, int i) {
  const int u = g.i0 + i;
  return u < g.gap_at ? u : u + g.gap;
}

// A block's walk over its part of the list, an entry at a time. P holds the call's sizes (B,
// kv_heads, tile_tokens, window, sinks) and gives the new tokens [lo, hi) and the length of
// request b by request(b, lo, hi).
struct AttWalk {
  int skip, end;   // places of the list given out, and where the part ends
  int rest;        // places of the current unit given out
  int total, blocks, b, lo, hi, len, head, u, q_at;
  int lo1, hi1, len1;  // request b + 1, read ahead
  unsigned ring;
  AttJoin join;

  // The part [begin, end_), begin < end_, starts in request b_ (rows lo_ .. hi_ - 1, length
  // len_), before which there are `before` tiles.
  template <typename P>
  SV_LIST void start(const P& p, int begin, int end_, int total_, int blocks_, int b_, int before,
                     int lo_, int hi_, int len_) {
    lo = lo_, hi = hi_, len = len_;
    skip = begin, end = end_, total = total_, blocks = blocks_, b = b_;
    u = q_at = 0;
    ring = 0;
    join = {-1, 0, 0, 0};
    read_ahead(p);
    const AttUnits units(len, hi - lo, 2 * p.tile_tokens, p.window, p.sinks);
    const int x = begin - before;
    head = rest = 0;
    if (x == 0) return;
    const int per_head = units.before(units.count);
    head = x / per_head;
    rest = x - head * per_head;
    int u1 = units.count - 1;  // the last unit that starts at or before there
    while (u < u1) {
      const int mid = (u + u1 + 1) >> 1;
      if (units.before(mid) <= rest) u = mid; else u1 = mid - 1;
    }
    rest -= units.before(u);
  }
  template <typename P>
  SV_LIST void read_ahead(const P& p) {
    if (b + 1 < p.B) len1 = p.request(b + 1, lo1, hi1);
  }

  template <typename P>
  SV_LIST void next_request(const P& p) {
    lo = lo1, hi = hi1, len = len1;
    read_ahead(p);
  }

  // The next entry; g.n = 0 past the last.
  template <typename P>
  SV_LIST void next(const P& p, AttSeg& g) {
    const int step = 2 * p.tile_tokens;
    g.n = 0;
    // A unit takes its key tiles and `cost` places more in the list, which stand for what its
    // start and its results cost.
    while (skip < end) {
      while (hi == lo && b + 1 < p.B) {  // requests without rows
        ++b;
        next_request(p);
      }
      const AttUnits units(len, hi - lo, step, p.window, p.sinks);
      const int n = units.tiles(u), here = min(n + units.cost - rest, end - skip);
      const int take = min(n - rest, here);  // tiles among them
      if (take > 0) {
        g.n = take;
        g.i0 = rest;
        g.b = b;
        g.head = head;
        g.token = lo + u * step;
        g.tokens = min(step, hi - g.token);
        g.pos = units.p0 + u * step;
        g.lo = units.lo(u);
        g.hi = max(units.hi(u), 0);
        g.gap = units.gap(u);
        g.gap_at = g.gap ? units.sink_tiles : 0x7fffffff;
        g.pair = g.tokens > p.tile_tokens;
        g.q_at = q_at;
        g.ring = ring;
        const bool starts = rest == 0, ends = rest + take == n;
        g.slot = starts && ends ? -1 : starts ? 1 : 0;
        if (starts && !ends) {
          join.last = att_block_of(skip + n - 1, total, blocks);
          join.head = head;
          join.token = g.token;
          join.tokens = g.tokens;
        }
        q_at += g.pair ? 2 : 1;
        ring += 2 * take;
      }
      skip += here;
      rest += here;
      if (rest == n + units.cost) {
        rest = 0;
        if (++u == units.count) {
          u = 0;
          if (++head == p.kv_heads) {
            head = 0;
            ++b;
            next_request(p);
          }
        }
      }
      if (take > 0) break;
    }
  }
};

}  // namespace sv
