// The closed forms of tq_chunk_cost.h against plain walks over tiles, and how often
// the search for a place on the line asks for a sum. Prints one line a check; exits
// non-zero on the first failure. Plain C++, no GPU.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "tq_chunk_cost.h"

using namespace tq;

static std::mt19937 rng(7);
static int between(int a, int b) { return a + static_cast<int>(rng() % static_cast<unsigned>(b - a + 1)); }

// A unit's cost by its definition, position by position.
static long long cost_of(const ChunkSize& c, const ChunkCall& k, int j) {
  const long long q0 = 1ll * j * k.per;
  if (q0 >= c.served) return 0;
  const long long q1 = q0 + k.per < c.served ? q0 + k.per : c.served;
  long long seen = c.first + q1;
  if (seen > k.limit) seen = k.limit;
  long long steps = seen > 0 ? (seen + 127) / 128 : 0;
  if (steps < 1) steps = 1;
  return steps * ((c.served - q0) * k.group > k.full_rows ? 4 : 3) + 10;
}

static ChunkCall call_of(int group, int ctas, int limit) { return {ctas * 256 / group, limit, group, ctas * 128}; }

int main() {
  long long checks = 0;
  for (int round = 0; round < 4000; ++round) {
    const ChunkCall k = call_of(between(1, 8), between(1, 2), round % 5 == 0 ? between(0, 200) : between(1, 40000));
    const int far = round % 3 == 0 ? 20000 : 600;
    const ChunkSize c = {between(-far, far), between(0, far)};
    long long sum = 0;
    const int tiles = chunk_tiles(c, k.per);
    for (int j = 0; j <= tiles + 2; ++j, ++checks) {
      if (chunk_cost_before(c, k, j) != sum || static_cast<long long>(chunk_cost(c, k, j)) != cost_of(c, k, j) ||
          (chunk_cost(c, k, j) != 0) != (j < tiles)) {
        std::printf("FAIL tile %d of %d queries from position %d: per %d limit %d: %lld, %lld\n", j, c.served, c.first, k.per, k.limit,
                    chunk_cost_before(c, k, j), sum);
        return 1;
      }
      sum += cost_of(c, k, j);
    }
  }
  std::printf("costs %lld\n", checks);

  // far positions, where the sums pass 32 bits
  for (int group = 1; group <= 8; ++group) {
    const ChunkCall k = call_of(group, 2, 0x7fffff00);
    const ChunkSize c = {2000000000, 3000000};
    long long sum = 0;
    const int tiles = chunk_tiles(c, k.per);
    for (int j = 0; j < tiles; ++j) sum += cost_of(c, k, j);
    if (chunk_cost_before(c, k, tiles) != sum || sum >> 32 == 0) {
      std::printf("FAIL far positions, group %d: %lld, %lld\n", group, chunk_cost_before(c, k, tiles), sum);
      return 1;
    }
  }
  std::printf("far\n");

  // places on the line of many sequences: where a walk finds them, by few sums
  for (int round = 0; round < 300; ++round) {
    const ChunkCall k = call_of(between(1, 8), between(1, 2), 50000);
    std::vector<ChunkSize> all(between(1, 40));
    int end = 0;
    for (auto& c : all) {
      c = {between(0, 3000), between(0, 9) ? between(0, 5) : between(0, 9000)};
      if (chunk_tiles(c, k.per) > end) end = chunk_tiles(c, k.per);
    }
    int asked = 0;
    auto before = [&](int j) {
      ++asked;
      long long sum = 0;
      for (const auto& c : all) sum += chunk_cost_before(c, k, j);
      return sum;
    };
    const long long total = before(end);
    int log2 = 0;
    while (1 << log2 < end + 1) ++log2;
    for (int i = 0; i < 20 && total; ++i) {
      const long long x = (static_cast<long long>(rng()) << 20 ^ rng()) % total;
      int j = 0, want = 0;
      long long base = 0, sum = 0;
      for (;; ++want) {
        long long here = 0;
        for (const auto& c : all) here += cost_of(c, k, want);
        if (x < sum + here) break;
        sum += here;
      }
      asked = 0;
      chunk_seek(x, end, 1, false, j, base, before);
      if (j != want || base != sum || asked > log2) {
        std::printf("FAIL place %lld of %lld: tile %d (%lld) for %d (%lld), %d sums\n", x, total, j, base, want, sum, asked);
        return 1;
      }
      // from a place before it on
      int from = want > 0 ? between(0, want) : 0;
      base = before(from);
      asked = 0;
      chunk_seek(x, end, 1, true, from, base, before);
      if (from != want || base != sum || asked > 2 * log2 + 1) {
        std::printf("FAIL place %lld from a place before it: tile %d for %d, %d sums\n", x, from, want, asked);
        return 1;
      }
      // down to a few
      for (int near = 0; near < 2; ++near) {
        const int close = between(2, 9);
        from = want > 0 ? between(0, want) : 0;
        base = before(from);
        asked = 0;
        chunk_seek(x, end, close, near, from, base, before);
        if (from > want || from + close <= want || base != before(from) || asked - 1 > 2 * log2 + 1) {
          std::printf("FAIL place %lld: tiles %d and %d more, without %d\n", x, from, close - 1, want);
          return 1;
        }
      }
    }
  }
  std::printf("places\n");

  // 4095 sequences of one query and one of 131072, 8 heads: sums over 128 groups of 32 sequences that both ends of a
  // part ask for, at most
  {
    const ChunkCall k = call_of(8, 2, 131072);
    const ChunkSize c = {0, 131072};
    int asked = 0, most = 0;
    auto before = [&](int j) {
      ++asked;
      return chunk_cost_before(c, k, j) + (j > 0 ? 4095 * 13ll : 0);
    };
    const int end = chunk_tiles(c, k.per);
    const long long total = before(end);
    for (int team = 0; team < 76; ++team) {
      int j = 0;
      long long base = 0;
      asked = 0;
      chunk_seek(total * team / 76, end, 8, false, j, base, before);
      if (team < 75) chunk_seek(total * (team + 1) / 76, end, 8, true, j, base, before);
      if (asked > most) most = asked;
    }
    if (end != 2048 || most > 3 * 8 + 1) {
      std::printf("FAIL %d tiles, %d sums\n", end, most);
      return 1;
    }
    std::printf("sums %d\n", most);
  }
  return 0;
}
