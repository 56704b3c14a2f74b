// The list of key tiles and a block's walk over it (attend_list.cuh) as plain C++,
// for test_attend_list.py.
#include "../speculative_decoding_rejection_02_gb300/csrc/attend_list.cuh"

#include <cstring>
#include <new>
#include <vector>

namespace {

struct Call {
  int B, kv_heads, tile_tokens, window, sinks;
  const int *cu_q, *kv_lens;
  int request(int b, int& lo, int& hi) const {
    lo = cu_q[b];
    hi = cu_q[b + 1];
    return kv_lens[b];
  }
};

}  // namespace

extern "C" {

long long list_before(int len, int q, int step, int window, int sinks, int k) {
  return sv::AttUnits(len, q, step, window, sinks).before(k);
}

// Walks the parts of all blocks. Entry i of block c is segs[first[c] + i]; first has blocks + 1
// entries. Returns the number of blocks with a part, -1 where `most` entries are too few.
int list_walk(const int* cu_q, const int* kv_lens, int B, int kv_heads, int tile_tokens,
              int window, int sinks, int grid, sv::AttSeg* segs, long long most, long long* first,
              sv::AttJoin* joins) {
  const Call p = {B, kv_heads, tile_tokens, window, sinks, cu_q, kv_lens};
  std::vector<long long> before(B + 1, 0);
  for (int b = 0; b < B; ++b) {
    const sv::AttUnits units(kv_lens[b], cu_q[b + 1] - cu_q[b], 2 * tile_tokens, window, sinks);
    before[b + 1] = before[b] + (long long)units.before(units.count) * kv_heads;
  }
  const long long total = before[B];
  const int blocks = total < grid ? (int)total : grid;
  long long at = 0;
  int b = 0;
  first[0] = 0;
  for (int c = 0; c < blocks; ++c) {
    const sv::AttPart part(c, total, blocks);
    while (before[b + 1] <= part.begin) ++b;
    alignas(sv::AttWalk) unsigned char memory[sizeof(sv::AttWalk)];
    std::memset(memory, 0xcd, sizeof memory);  // the walk has to set all that next() reads
    sv::AttWalk& walk = *new (memory)
        sv::AttWalk(p, part, c, b, before[b], cu_q[b], cu_q[b + 1], kv_lens[b]);
    for (;; ++at) {
      if (at == most) return -1;
      walk.next(p, segs[at]);
      if (segs[at].n == 0) break;
    }
    joins[c] = walk.join;
    first[c + 1] = at;
  }
  return blocks;
}

}  // extern "C"
