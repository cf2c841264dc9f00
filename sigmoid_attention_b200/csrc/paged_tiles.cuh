// paged_tiles.cuh -- how many key blocks the query tiles of a sequence walk: the
// units that paged_run.cuh shares out. (Plain arithmetic: it compiles for the host
// too, where a test compares it with sums over all tiles.)
#pragma once

#include <cstdint>

namespace sigattn {

constexpr int kKeyBlock = 128;

// Key blocks that a tile seeing n keys walks (one even without keys: its rows
// are written as zeros).
__device__ __forceinline__ int seq_blocks(int n) { return n > 0 ? (n + kKeyBlock - 1) / kKeyBlock : 1; }

// A sequence's first row, new tokens m and cached tokens n.
struct SeqInfo {
  int start, m, n;
};

// sum_{k < n} floor((x k + y) / 128), x n and y less than 2^25. Where x is a power
// of two (G is one) the sum has a closed form; otherwise by the Euclid-like
// algorithm for such sums: after taking out whole parts, the lattice points under
// the line are counted along the other axis.
template <typename U>
__device__ __forceinline__ U floor_sum(uint32_t n, uint32_t x, uint32_t y) {
  // Half of an even product (halved first: U may hold the sum but not its terms,
  // which is harmless where each step is exact modulo its size).
  auto half = [](uint32_t v, uint32_t w) { return (v & 1) ? static_cast<U>(v) * (w >> 1) : static_cast<U>(v >> 1) * w; };
  if ((x & (x - 1)) == 0) {
    const int e = 31 - __clz(x);
    if (e >= 7) return (half(n, n - 1) << (e - 7)) + static_cast<U>(n) * (y >> 7);
    const int f = 7 - e;  // floor((x k + y) / 128) = floor((k + (y >> e)) / 2^f)
    auto upto = [&](uint32_t k) {
      const uint32_t t = k >> f;
      return (half(t, t - 1) << f) + static_cast<U>(t) * (k & ((1u << f) - 1));
    };
    return upto((y >> e) + n) - upto(y >> e);
  }
  uint32_t m = kKeyBlock;
  U sum = 0;
  while (n > 0) {
    if (x >= m) {
      const uint32_t q = x / m;
      sum += half(n, n - 1) * q;
      x -= q * m;
    }
    if (y >= m) {
      const uint32_t q = y / m;
      sum += static_cast<U>(n) * q;
      y -= q * m;
    }
    const uint32_t top = x * n + y;
    if (top < m) break;
    n = top / m;
    y = top - n * m;
    const uint32_t t = m;
    m = x;
    x = t;
  }
  return sum;
}

// paged_many.cu: a sequence's tiles. An item is two query tiles, 2 T tokens (the
// last may be one), or one tile where the call has few and short ones
// (kLoneUnits): more CTAs then share the tiles, their parts and the adding up of
// these, at the cost of loading each key block once per tile. A block of an item is
// as many units as it has tiles: two tiles' products bound a block, one tile's are
// about as fast as its keys arrive, in half the time.
struct TileMath {
  int T;
  int pairs;  // items of two tiles
  int causal;
  __device__ __forceinline__ int item() const { return T << pairs; }
  __device__ __forceinline__ int items(const SeqInfo& s) const { return (s.m + item() - 1) / item(); }
  __device__ __forceinline__ bool two(int m, int k) const { return pairs && k * 2 * T + T < m; }
  __device__ __forceinline__ bool two(const SeqInfo& s, int k) const { return two(s.m, k); }
  __device__ __forceinline__ int shift(const SeqInfo& s, int k) const { return two(s, k) ? 1 : 0; }
  // Keys that token i sees.
  __device__ __forceinline__ int seen(int m, int n, int i) const {
    return causal ? max(0, min(n, n - m + i + 1)) : n;
  }
  // Blocks that tokens up to i of the chunk walk.
  __device__ __forceinline__ int blocks(int m, int n, int i) const { return seq_blocks(seen(m, n, i)); }
  __device__ __forceinline__ int blocks(const SeqInfo& s, int k) const {
    return blocks(s.m, s.n, min((k + 1) * item(), s.m) - 1);
  }
  // Units of items 0 .. k - 1 (k <= items).
  template <typename U>
  __device__ __forceinline__ U before(const SeqInfo& s, int k) const {
    U sum = 0;
    if (k > 0 && k == items(s)) {  // the last item may hold fewer tokens
      --k;
      sum = static_cast<U>(seq_blocks(s.n)) << shift(s, k);
    }
    if (!causal) return sum + (static_cast<U>(k) * seq_blocks(s.n) << pairs);
    // Item i's last token sees n - m + (i + 1) 2 T keys, or (more rows than
    // tokens) none: then it still walks the block that writes its zeros.
    const int item = this->item(), c = s.n - s.m;
    const int none = c < 0 ? min(k, -c / item) : 0;
    return sum + ((static_cast<U>(none) + floor_sum<U>(k - none, item, c + (none + 1) * item + kKeyBlock - 1)) << pairs);
  }
};

// paged_few.cu: all new tokens of a sequence make one tile.
struct OneTile {
  __device__ __forceinline__ int items(const SeqInfo&) const { return 1; }
  __device__ __forceinline__ int blocks(const SeqInfo& s, int) const { return seq_blocks(s.n); }
  __device__ __forceinline__ int shift(const SeqInfo&, int) const { return 0; }
  template <typename U>
  __device__ __forceinline__ U before(const SeqInfo& s, int k) const {
    return static_cast<U>(k) * seq_blocks(s.n);
  }
};

}  // namespace sigattn
