// What the chunks of tq_kv16_continue cost, in closed form: host and device, no
// CUDA needed. Internal, not ABI.
//
// A sequence's chunk has tiles of `per` queries; tile j sees the positions up to
// its last query's, at most `limit`, in steps of 128. A unit (a tile, one KV head)
// costs 4 a step, or 3 where one of its two row tiles is at work, and 10 more
// (1.45, 1.14 and 3 to 4 us). Steps grow linearly in j up to `limit`, so what the
// tiles before j cost together needs no walk over them; a place on the line of all
// units is found by bisection over j, and a walk over the last few.
#ifndef TQ_CHUNK_COST_H_
#define TQ_CHUNK_COST_H_

#ifdef __CUDACC__
#define TQ_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define TQ_HOST_DEVICE inline
#endif

namespace tq {

constexpr int kChunkCols = 128;       // positions a step
constexpr unsigned kChunkUnit = 10;   // of a unit, beyond its steps

// A chunk: the position of its first query (negative: it has more queries than positions), queries that are served.
struct ChunkSize {
  int first, served;
};
// The call: queries a tile, positions at most, heads, and the rows of a unit above which both row tiles are at work.
struct ChunkCall {
  int per, limit, group, full_rows;
};

TQ_HOST_DEVICE int chunk_min(int x, int y) { return x < y ? x : y; }
TQ_HOST_DEVICE int chunk_max(int x, int y) { return x > y ? x : y; }

TQ_HOST_DEVICE int chunk_tiles(const ChunkSize& c, int per) { return static_cast<int>(static_cast<unsigned>(c.served + per - 1) / static_cast<unsigned>(per)); }
// Positions that the last query of tile j sees.
TQ_HOST_DEVICE int chunk_limit(const ChunkSize& c, const ChunkCall& k, int j) {
  return chunk_max(chunk_min(c.first + chunk_min((j + 1) * k.per, c.served), k.limit), 0);
}
// The steps of a unit of tile j: one at least, though it may see nothing; 0 if there is no such tile.
TQ_HOST_DEVICE int chunk_steps(const ChunkSize& c, const ChunkCall& k, int j) {
  return j * k.per < c.served ? chunk_max((chunk_limit(c, k, j) + kChunkCols - 1) / kChunkCols, 1) : 0;
}
TQ_HOST_DEVICE int chunk_each(const ChunkSize& c, const ChunkCall& k, int j) { return (c.served - j * k.per) * k.group > k.full_rows ? 4 : 3; }
TQ_HOST_DEVICE unsigned chunk_cost(const ChunkSize& c, const ChunkCall& k, int j) {
  const int s = chunk_steps(c, k, j);
  return s ? static_cast<unsigned>(s) * chunk_each(c, k, j) + kChunkUnit : 0u;
}

// sum over i = 1 .. m of floor((r + i c) / 128), 0 <= r, c < 128: the sum of the numbers less that of their remainders,
// which repeat after 128 / g, g the largest power of two in c, and over that many are r % g, r % g + g, .. once each.
TQ_HOST_DEVICE long long chunk_floors(unsigned m, unsigned c, unsigned r) {
  if (c == 0) return 0;
  const unsigned g = c & (0u - c), period = 128u / g;
  const long long n = m;
  long long left = n / period * (period * (r & (g - 1)) + 64u * (period - 1));
  unsigned x = r;
  for (unsigned i = m % period; i; --i) {
    x = (x + c) & 127u;
    left += x;
  }
  return (n * r + c * (n * (n + 1) / 2) - left) >> 7;
}

// The steps of the tiles before tile m, all of them full (m < the chunk's tiles).
TQ_HOST_DEVICE long long chunk_steps_before(const ChunkSize& c, const ChunkCall& k, int m) {
  if (m <= 0) return 0;
  // tile i - 1 sees first + i per: the first `low` tiles see 128 or less, those past `mid` all of `limit`
  const int low = chunk_max(chunk_min((kChunkCols - c.first) / k.per, m), 0);
  const int mid = chunk_max(chunk_min((k.limit - 1 - c.first) / k.per, m), low);
  long long sum = low + static_cast<long long>(m - mid) * chunk_max((k.limit + kChunkCols - 1) / kChunkCols, 1);
  if (mid > low) {
    const long long n = mid - low;
    const int at = c.first + low * k.per + kChunkCols - 1;   // > 0 with one tile more
    sum += n * (at >> 7) + (k.per >> 7) * (n * (n + 1) / 2) + chunk_floors(static_cast<unsigned>(n), k.per & 127, at & 127);
  }
  return sum;
}
// What the tiles before tile j cost, for one KV head; j from the chunk's tiles on: what all do.
TQ_HOST_DEVICE long long chunk_cost_before(const ChunkSize& c, const ChunkCall& k, int j) {
  if (c.served <= 0) return 0;
  const int tiles = chunk_tiles(c, k.per), m = chunk_min(j, tiles - 1);   // the full tiles among them cost 4 a step
  return 4 * chunk_steps_before(c, k, m) + static_cast<long long>(kChunkUnit) * m + (j >= tiles ? chunk_cost(c, k, tiles - 1) : 0u);
}

// Narrows down the tile index whose part of the line place x is in, the last j with before(j) <= x, to j .. j + close - 1:
// so few are walked sooner. In: a j at or before it, with base = before(j), and an `end` with before(end) > x. near: most
// likely close to j (else anywhere).
template <typename Before>
TQ_HOST_DEVICE void chunk_seek(long long x, int end, int close, bool near, int& j, long long& base, Before&& before) {
  int ahead = near ? close : 0;   // how far to look: twice as far each time, until that is too far; then by halves
  while (end - j > close) {
    const int mid = ahead && ahead < end - j ? j + ahead : j + (end - j) / 2;
    const long long here = before(mid);
    if (here <= x) {
      j = mid;
      base = here;
      ahead *= 2;
    } else {
      end = mid;
      ahead = 0;
    }
  }
}

}  // namespace tq

#endif  // TQ_CHUNK_COST_H_
