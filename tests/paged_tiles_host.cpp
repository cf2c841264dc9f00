// The planning arithmetic of the paged attention kernels, compiled for the host.
// Reads lines "T pairs causal m n k", writes the units before item k in 32 and
// in 64 bits, and its blocks and shift.
#include <algorithm>
#include <cstdio>

#define __device__
#define __forceinline__ inline
static int __clz(unsigned x) { return x ? __builtin_clz(x) : 32; }
using std::max;
using std::min;
#include "../sigmoid_attention_b200/csrc/paged_tiles.cuh"

int main() {
  int T, pairs, causal, m, n, k;
  while (std::scanf("%d %d %d %d %d %d", &T, &pairs, &causal, &m, &n, &k) == 6) {
    const sigattn::TileMath math{T, pairs, causal};
    const sigattn::SeqInfo s{0, m, n};
    const int item = min(k, math.items(s) - 1);
    std::printf("%u %llu %d %d %d\n", math.before<uint32_t>(s, k), math.before<unsigned long long>(s, k), math.items(s),
                math.blocks(s, item), math.shift(s, item));
  }
  return 0;
}
