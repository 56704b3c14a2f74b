// The list of key tiles that an attention call works through (cache_attend.cuh),
// and a block's walk over its part of it: arithmetic alone, which also compiles
// as plain C++ for the tests.
//
// A unit is up to two tiles of rows of one request and kv head. It takes its key
// tiles and a fixed number of places more, which stand for what its start and its
// results cost. The list is all units in order of request, kv head and rows, and
// is never written down: a block finds its part from the requests' lengths. A list
// may be longer than 2^32 places (a chunk of 1.6 million tokens in units of two has
// 5e9), a block's part of it may not (kAttMostPart).
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
// The most places of a block's part: its loads are counted in 32 bits, two for each place.
// (That many take a block about ten minutes.)
constexpr long long kAttMostPart = 1ll << 30;

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

// sum over 0 <= u < n of floor((a u + b) / kAttTile), a <= 2 kAttTile, b <= 2^31: n may be so
// large that the sum needs 64 bits. A term is a more than the one kAttTile before it, and the
// kAttTile terms of one such period together need only 32.
SV_LIST long long tile_sum(unsigned n, unsigned a, unsigned b) {
  const unsigned periods = n / kAttTile, rest = n % kAttTile;
  const long long rise = (long long)a * periods;  // of a term over all periods
  long long sum = rise * rest + rise * (kAttTile / 2) * (periods - (periods > 0));
#ifdef __CUDACC__
#pragma unroll 1
#endif
  for (int whole = 0; whole <= (periods > 0); ++whole)
    sum += (long long)floor_sum(whole ? kAttTile : rest, kAttTile, a, b) * (whole ? periods : 1);
  return sum;
}

// The units of one request: `count` of `step` new tokens each (the last may
// have fewer), for each kv head. Positions are below 2^31.
struct AttUnits {
  int p0;  // position of the first new token
  int q, step, count, window, sink_tiles, cost;

  SV_LIST AttUnits(int len, int q_, int step_, int window_, int sinks)
      : p0(len - q_), q(q_), step(step_), count(q_ <= step_ ? q_ > 0 : (q_ - 1) / step_ + 1),
        window(window_), sink_tiles((int)(((unsigned)sinks + kAttTile - 1) / kAttTile)),
        cost(q_ > step_ / 2 ? kAttPairCost : kAttCost) {}

  SV_LIST int hi(int u) const {
    return p0 + (u + 1 < count ? (u + 1) * step : q);
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
  SV_LIST long long before(int k) const {
    long long sum = (long long)k * cost;
    if (k == count && k > 0) sum += tiles(--k);  // the last one ends where the request does
    if (k <= 0) return sum;
    int dead = p0 < 0 ? -p0 / step : 0;  // units before position 0
    if (dead > k) dead = k;
    if (dead < k)
      sum += tile_sum(k - dead, step, (unsigned)p0 + (dead + 1) * step + kAttTile - 1);
    sum += dead;
    if (window) {
      const long long from =
          (long long)(sink_tiles + 1) * kAttTile + window - 1 - p0;  // gap > 0
      const long long u = from > 0 ? (from + step - 1) / step : 0;
      if (u < k)
        sum -= tile_sum(k - (int)u, step, (unsigned)(p0 + u * step - window + 1)) -
               (k - u) * sink_tiles;
    }
    return sum;
  }
};

// One block's part of the list: the first total % blocks parts are a place longer.
struct AttPart {
  long long begin;
  int places;
  int part, longer;  // places of the later parts, of which the first `longer` have one more

  // Of block c of blocks <= 2^16 with 0 < total <= kAttMostPart * blocks.
  SV_LIST AttPart(int c, long long total, unsigned blocks) {
    // total / blocks in two steps of 32 bits (a division of 64 is a long call)
    const unsigned high = (unsigned)(total >> 16);
    const unsigned low = (high % blocks) << 16 | ((unsigned)total & 0xffff);
    const unsigned more = low % blocks;
    part = (int)((high / blocks << 16) + low / blocks);
    begin = (long long)c * part + min((unsigned)c, more);
    places = part + ((unsigned)c < more);
    longer = max((int)more - c - 1, 0);
  }
  // How many blocks later the place lies that is `x` places past the part's end.
  SV_LIST int blocks_to(int x) const {
    if (x < (long long)longer * (part + 1)) return 1 + x / (part + 1);
    return 1 + longer + (x - longer * (part + 1)) / part;
  }
};

// Number of the entry's key tile i.
SV_LIST int att_tile(const AttSeg& g, int i) {
  const int u = g.i0 + i;
  return u < g.gap_at ? u : u + g.gap;
}

// A block's walk over its part of the list, an entry at a time. P holds the call's sizes (B,
// kv_heads, tile_tokens, window, sinks) and gives the new tokens [lo, hi) and the length of
// request b by request(b, lo, hi).
struct AttWalk {
  AttPart part;
  int left;        // places of the part not given out
  int rest;        // places of the current unit given out
  int block, b, lo, hi, len, head, u, q_at;
  int lo1, hi1, len1;  // request b + 1, read ahead
  unsigned ring;
  AttJoin join;

  // The part of block block_ starts in request b_ (rows lo_ .. hi_ - 1, length len_), before
  // which there are `before` places.
  template <typename P>
  SV_LIST AttWalk(const P& p, const AttPart& part_, int block_, int b_, long long before, int lo_,
                  int hi_, int len_)
      : part(part_), left(part_.places), rest(0), block(block_), b(b_), lo(lo_), hi(hi_),
        len(len_), head(0), u(0), q_at(0), ring(0), join{-1, 0, 0, 0} {
    read_ahead(p);
    const AttUnits units(len, hi - lo, 2 * p.tile_tokens, p.window, p.sinks);
    const long long x = part.begin - before;
    if (x == 0) return;
    // The head, from the length of a whole one; then the last unit of it that starts at or
    // before the part. (One loop, so that before()'s code is there once.)
    long long in_head = 0, from = 0;
    int u1 = units.count - 1;
    for (int k = units.count;;) {
      const long long at = units.before(k);
      if (k == units.count) {
        head = (int)(x / at);
        in_head = x - head * at;
      } else if (at <= in_head) {
        u = k;
        from = at;
      } else {
        u1 = k - 1;
      }
      if (u >= u1) break;
      k = (u + u1 + 1) >> 1;
    }
    rest = (int)(in_head - from);
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
    while (left > 0) {
      while (hi == lo && b + 1 < p.B) {  // requests without rows
        ++b;
        next_request(p);
      }
      const AttUnits units(len, hi - lo, step, p.window, p.sinks);
      const int n = units.tiles(u), here = min(n + units.cost - rest, left);
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
          join.last = block + part.blocks_to(n - here - 1);
          join.head = head;
          join.token = g.token;
          join.tokens = g.tokens;
        }
        q_at += g.pair ? 2 : 1;
        ring += 2 * take;
      }
      left -= here;
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
