// paged_run.cuh -- how the paged attention kernels share a call's work out.
//
// A call's units of work (blocks of 128 keys of one query tile of one key/value
// head of one sequence) stand in one line: sequences in batch order, heads,
// tiles, blocks. The line is cut into equal runs, one per CTA. Each CTA finds
// its run itself (plan_run: a prefix sum over the batch's lengths), its
// producer walks it and hands every segment (the part of one tile's blocks
// that lies in the run) to the other roles through a ring in shared memory.
// A tile whose blocks lie in several CTAs is joined by the CTA that stores
// its part last (last_part).
// Blocks may weigh 1 or 2 units (a block for one query tile or for two); a block
// belongs to the CTA in whose run its first unit lies.
#pragma once

#include <climits>

#include "paged.cuh"

namespace sigattn {

constexpr int kKeyBlock = 128;

// Key blocks that a tile seeing n keys walks (one even without keys: its rows
// are written as zeros).
__device__ __forceinline__ int seq_blocks(int n) { return n > 0 ? (n + kKeyBlock - 1) / kKeyBlock : 1; }

// A wait by a whole warp: every lane gets the same answer, so that an aborting
// warp leaves its loop as one.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* ws, int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, ws, site));
}

// (The lengths and tables below are loaded from L2: the kernel before this one
// may write them while this one's CTAs are already resident.)
// Sequence b's first row, new tokens m and cached tokens n; false (and m = 0)
// if it breaks the call's rules.
struct SeqInfo {
  int start, m, n;
};
// (as loaded: loads are issued ahead and checked when they are needed)
struct SeqWords {
  int start, end, n;
};
__device__ __forceinline__ SeqWords seq_load(const PagedAttend& a, int b) {
  b = min(b, a.B - 1);
  return SeqWords{__ldcg(a.cu + b), __ldcg(a.cu + b + 1), __ldcg(a.kv + b)};
}
__device__ __forceinline__ bool seq_check(const PagedAttend& a, const SeqWords& w, SeqInfo* s) {
  const bool ok = w.start >= 0 && w.end >= w.start && w.end <= a.total && w.end - w.start <= a.max_q && w.n >= 0 &&
                  w.n <= a.max_pages << a.page_shift;
  s->start = w.start;
  s->m = ok ? w.end - w.start : 0;
  s->n = w.n;
  return ok;
}

// x / y of nonnegative numbers: unit counts nearly always fit 32 bits, where a
// division takes a fraction of the time.
__device__ __forceinline__ long long fast_div(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// A CTA's run: `count` units from unit blockIdx.x * per of the line on, which is
// unit `rem` of sequence b.
struct PlanRun {
  long long rem;
  SeqInfo s;
  int b, count, per;
};

// units(s): units of one key/value head of a sequence with new tokens. Runs are
// at least a.least units long (at least a block's weight, so that a tile's CTAs
// all have a block of it).
// Ends before the caller's next barrier; every thread of the CTA takes part.
template <int THREADS, typename Units>
__device__ __forceinline__ void plan_run(const PagedAttend& a, PlanRun* run, Units units) {
  static_assert(THREADS % 32 == 0, "whole warps");
  __shared__ long long sums[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = ceil_div(a.B, THREADS);
  const int b0 = min(a.B, tid * chunk), b1 = min(a.B, b0 + chunk);
  SeqInfo s;  // of the sequence that units_of saw last
  auto units_of = [&](int b, bool report) -> long long {
    if (!seq_check(a, seq_load(a, b), &s)) {
      if (report && blockIdx.x == 0) raise_invalid(a.ws, -(b + 1));
      return 0;
    }
    return s.m > 0 ? static_cast<long long>(units(s)) * a.Hkv : 0;
  };
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += units_of(b, true);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  long long base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) base = total;
    total += sums[w];
  }
  base += incl - mine;
  long long per = max(static_cast<long long>(a.least), fast_div(total + gridDim.x - 1, gridDim.x));
  if (per > INT_MAX) {  // beyond any call that could end
    if (blockIdx.x == 0 && tid == 0) raise_invalid(a.ws, 206);
    per = total = 0;
  }
  const long long first = min(total, per * blockIdx.x);
  if (tid == 0) {
    run->count = static_cast<int>(min(per, total - first));
    run->per = static_cast<int>(per);
  }
  if (first >= base && first < base + mine) {
    long long rem = first - base;
    int b = b0;
    for (; chunk > 1; ++b) {  // (a thread with one sequence still holds it)
      const long long u = units_of(b, false);
      if (rem < u) break;
      rem -= u;
    }
    run->b = b;
    run->rem = rem;
    run->s = s;
  }
}

// Part of one tile's key blocks: blocks [j0, j1) of `blocks`. The tile's first
// and last blocks lie in CTAs first_cta and last_cta, its first unit is unit
// `lead` of first_cta's run. j1 < 0 ends a run.
struct Segment {
  int start, m, n, b;
  int head, tile, j0, j1;
  int blocks, first_cta, last_cta, lead;
};
static_assert(sizeof(Segment) == 48, "three int4");

// The first block of the tile that the p-th CTA after first_cta works on.
__device__ __forceinline__ int part_begin(const Segment& s, int p, int per, int weight) {
  return p == 0 ? 0 : static_cast<int>((static_cast<long long>(p) * per - s.lead + weight - 1) / weight);
}

__device__ __forceinline__ Segment end_segment() {
  Segment s{};
  s.j1 = -1;
  return s;
}

struct SegRing {
  static constexpr int kSlots = 4;
  int4 slot[kSlots][3];
  uint64_t full[kSlots], empty[kSlots];
};

__device__ __forceinline__ void seg_ring_init(SegRing& r, int consumers) {
  for (int s = 0; s < SegRing::kSlots; ++s) {
    mbar_init(&r.full[s], 1);
    mbar_init(&r.empty[s], consumers);
  }
}

// The whole producer warp calls this.
__device__ __forceinline__ bool seg_publish(SegRing& r, uint32_t& st, uint32_t& ph, const Segment& s, int lane,
                                            volatile int* abort_flag, int* ws, int site) {
  if (!warp_wait(&r.empty[st], ph ^ 1, abort_flag, ws, site)) return false;
  if (lane == 0) {
    r.slot[st][0] = make_int4(s.start, s.m, s.n, s.b);
    r.slot[st][1] = make_int4(s.head, s.tile, s.j0, s.j1);
    r.slot[st][2] = make_int4(s.blocks, s.first_cta, s.last_cta, s.lead);
    mbar_arrive(&r.full[st]);
  }
  __syncwarp();
  if (++st == SegRing::kSlots) { st = 0; ph ^= 1; }
  return true;
}

__device__ __forceinline__ Segment seg_peek(SegRing& r, uint32_t st) {
  const int4 x = r.slot[st][0], y = r.slot[st][1], z = r.slot[st][2];
  return Segment{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
}

// Wait for the next segment and copy it out; its slot stays taken until
// seg_release. WARP: a whole warp calls this (otherwise one thread of it).
template <bool WARP>
__device__ __forceinline__ bool seg_read(SegRing& r, uint32_t st, uint32_t ph, Segment* s, volatile int* abort_flag,
                                         int* ws, int site) {
  if (!(WARP ? warp_wait(&r.full[st], ph, abort_flag, ws, site) : mbar_wait(&r.full[st], ph, abort_flag, ws, site)))
    return false;
  *s = seg_peek(r, st);
  return true;
}

__device__ __forceinline__ void seg_release(SegRing& r, uint32_t& st, uint32_t& ph, bool arrive) {
  if (arrive) mbar_arrive(&r.empty[st]);
  if (++st == SegRing::kSlots) { st = 0; ph ^= 1; }
}

// A producer warp's walk along its CTA's run. Lengths and page numbers come from
// global memory: lane l holds the lengths of sequence base + l and the page
// of table entry window + l, and the next ones (the following 32 sequences, the
// following 32 entries, the next sequence's first 32 entries) are loaded long
// before they are needed, so that only the run's first block waits for them.
//
// Tiles: items(s), blocks(s, tile), a block's weight(s, tile) and before(s, k)
// (the units of tiles 0 .. k - 1) of one key/value head of a sequence with new
// tokens.
template <typename Tiles>
struct RunWalker {
  const PagedAttend& a;
  const Tiles& tiles;
  const int lane, per, count;
  int pos;     // units of the run up to the current segment's end
  bool alive;  // there is a current segment
  Segment seg;
  SeqInfo s, next_s;
  int items, next_b;
  int seq_base;
  SeqWords seq_cur, seq_ahead;
  const int* row;
  int pages, first, next_first, window, cur, ahead;

  // Find the next sequence after b with new tokens (a.B: none) and start the
  // load of its first page numbers.
  __device__ __forceinline__ void look_ahead(int b) {
    for (;;) {
      const int from = b + 1 - seq_base;  // 1 .. 32
      SeqInfo x;
      seq_check(a, seq_cur, &x);
      unsigned found = __ballot_sync(0xffffffffu, x.m > 0 && seq_base + lane < a.B);
      found = from < 32 ? found >> from << from : 0u;
      if (found) {
        const int l = __ffs(found) - 1;
        next_b = seq_base + l;
        next_s = SeqInfo{__shfl_sync(0xffffffffu, x.start, l), __shfl_sync(0xffffffffu, x.m, l),
                         __shfl_sync(0xffffffffu, x.n, l)};
        next_first = entry(a.table + static_cast<size_t>(next_b) * a.max_pages, pages_of(next_s.n), 0);
        return;
      }
      seq_base += 32;
      if (seq_base >= a.B) break;
      seq_cur = seq_ahead;
      seq_ahead = seq_load(a, seq_base + 32 + lane);
      b = seq_base - 1;
    }
    next_b = a.B;
  }
  __device__ __forceinline__ int pages_of(int n) const { return (n + (1 << a.page_shift) - 1) >> a.page_shift; }
  __device__ __forceinline__ int entry(const int* r, int limit, int i) const {
    return i + lane < limit ? __ldcg(r + i + lane) : -1;
  }
  __device__ __forceinline__ void enter() {
    seg.start = s.start;
    seg.m = s.m;
    seg.n = s.n;
    row = a.table + static_cast<size_t>(seg.b) * a.max_pages;
    pages = pages_of(s.n);
    items = tiles.items(s);
  }

  __device__ __forceinline__ RunWalker(const PagedAttend& args, const Tiles& t, const PlanRun& run, int ln)
      : a(args), tiles(t), lane(ln), per(run.per), count(run.count), pos(0), alive(run.count > 0) {
    if (!alive) return;
    s = run.s;
    seg = Segment{};
    seg.b = run.b;
    enter();
    first = entry(row, pages, 0);
    seq_base = seg.b;
    seq_cur = seq_load(a, seq_base + lane);
    seq_ahead = seq_load(a, seq_base + 32 + lane);
    next_b = -1;  // looked for when the run's first loads are on their way
    const long long each = tiles.before(s, items);
    seg.head = static_cast<int>(fast_div(run.rem, each));
    const long long rem = run.rem - seg.head * each;
    // The last tile with before(tile) <= rem, 32 candidates at a time.
    for (int width = items; width > 1;) {
      const int step = (width + 31) / 32;
      const unsigned below =
          __ballot_sync(0xffffffffu, lane * step < width && tiles.before(s, seg.tile + lane * step) <= rem);
      const int l = 31 - __clz(below);
      seg.tile += l * step;
      width = min(step, width - l * step);
    }
    seg.blocks = tiles.blocks(s, seg.tile);
    const int weight = tiles.weight(s, seg.tile), off = static_cast<int>(rem - tiles.before(s, seg.tile));
    seg.j0 = (off + weight - 1) / weight;
    pos = seg.j0 * weight - off;
    if (seg.j0 == seg.blocks) alive = step_tile();  // the run starts inside the tile's last block
    else open();
  }

  // The segment that starts at seg.j0, unit `pos` of the run. A tile that began
  // before it began in the run (only a run's first can); one that does not end
  // in it is its last.
  __device__ __forceinline__ void open() {
    const int me = blockIdx.x, weight = tiles.weight(s, seg.tile);
    const int len = min((count - pos + weight - 1) / weight, seg.blocks - seg.j0);
    const int begin = pos - seg.j0 * weight;  // where the tile begins, counted from the run's first unit
    seg.j1 = seg.j0 + len;
    seg.first_cta = me;
    seg.lead = begin;
    if (begin < 0) {
      const int back = (per - 1 - begin) / per;
      seg.first_cta = me - back;
      seg.lead = back * per + begin;
    }
    seg.last_cta = seg.j1 == seg.blocks ? me : me + (begin + (seg.blocks - 1) * weight) / per;
    pos += len * weight;
    window = ((seg.j0 * kKeyBlock) >> a.page_shift) & ~31;
    cur = window == 0 ? first : entry(row, pages, window);
    ahead = entry(row, pages, window + 32);
  }

  // On to the next tile; false at the run's end.
  __device__ __forceinline__ bool step_tile() {
    if (pos >= count) return false;
    seg.j0 = 0;
    if (next_b < 0) look_ahead(seg.b);
    if (++seg.tile == items) {
      seg.tile = 0;
      if (++seg.head == a.Hkv) {  // the next sequence
        seg.head = 0;
        if (next_b >= a.B) return false;
        s = next_s;
        seg.b = next_b;
        first = next_first;
        enter();
        look_ahead(seg.b);
      }
    }
    seg.blocks = tiles.blocks(s, seg.tile);
    open();
    return true;
  }
  __device__ __forceinline__ void next() { alive = step_tile(); }

  // Where box `box` (of rb keys) of block j lies: the slice (page * Hkv + head)
  // and *r, the row in it. A bad page (reported where `used`) lies past the last
  // slice, where a load reads zeros. Blocks come in order.
  __device__ __forceinline__ int locate(int j, int box, int rb, bool used, int* r) {
    if (((j * kKeyBlock) >> a.page_shift) >= window + 32) {
      window += 32;
      cur = ahead;
      ahead = entry(row, pages, window + 32);
    }
    const int key = j * kKeyBlock + box * rb;
    const int page = __shfl_sync(0xffffffffu, cur, (key >> a.page_shift) & 31);
    *r = key & ((1 << a.page_shift) - 1);
    if (page >= 0 && page < a.num_pages) return page * a.Hkv + seg.head;
    if (used) raise_invalid(a.ws, 203);
    return a.num_pages * a.Hkv;
  }
};

// After every epilogue warp of this CTA has stored its share of a tile's
// part: *last_flag tells whether this CTA's part was the tile's last (uniform over
// the CTA's epilogue warps; the other parts are then visible). `ph`: parity of
// the two barriers, flipped by the caller each time. The count of the tile's
// stored parts is one byte in the workspace header, put back to zero by the last.
__device__ __forceinline__ bool last_part(uint64_t* stored, uint64_t* counted, int* last_flag, const Segment& seg,
                                          int* ws, int warp, int lane, uint32_t ph, volatile int* abort_flag, int site) {
  // (The stores are ordered before the fence of warp 0's lane 0 by the barrier.)
  __syncwarp();
  if (lane == 0) mbar_arrive(stored);
  if (warp == 0) {
    if (!warp_wait(stored, ph, abort_flag, ws, site)) return false;
    if (lane == 0) {
      __threadfence();
      const int parts = seg.last_cta - seg.first_cta + 1;
      const int shift = 8 * (seg.first_cta & 3);
      unsigned* word = reinterpret_cast<unsigned*>(ws + kHdrParts + (seg.first_cta >> 2));
      const unsigned before = (atomicAdd(word, 1u << shift) >> shift) & 255u;
      const bool last = before == static_cast<unsigned>(parts - 1);
      if (last) atomicSub(word, static_cast<unsigned>(parts) << shift);
      __threadfence();
      *last_flag = last;
      mbar_arrive(counted);
    }
    __syncwarp();
  }
  return warp_wait(counted, ph, abort_flag, ws, site + 1);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace sigattn
