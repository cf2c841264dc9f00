// paged_run.cuh -- how the paged attention kernels share a call's work out.
//
// A call's work (the key blocks that the query tiles of each key/value head of
// each sequence walk) stands in one line: sequences in batch order, heads,
// tiles, blocks. The line is cut into equal runs, one per CTA. Each CTA finds
// its run itself (plan_run: a prefix sum over the batch's lengths), its
// producer walks it and hands every segment (the part of one tile's blocks
// that lies in the run) to the other roles through a ring in shared memory.
// A tile whose blocks lie in several CTAs is joined by the CTA that counts
// its part last (PartCount).
// Blocks are 1 or 2 units long (a block for one query tile or for two); a block
// belongs to the CTA in whose run its first unit lies. (Units of keys, so that
// texts' last blocks count by their keys, were tried: a short block takes as
// long as a full one, and 432 groups of 35 to 143 keys took 21 instead of 15 us.)
#pragma once

#include <climits>

#include "paged.cuh"
#include "paged_tiles.cuh"

namespace sigattn {

// mbar_wait with its slow path out of line: inlined at every wait, the clock and
// abort code made the roles' loops too long for the instruction cache.
static __device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* ws, int site) {
  return mbar_wait(bar, parity, abort_flag, ws, site);
}
__device__ __forceinline__ bool role_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* ws, int site) {
  return mbar_try_wait(bar, parity) || wait_longer(bar, parity, abort_flag, ws, site);
}

// A wait by a whole warp: every lane gets the same answer, so that an aborting
// warp leaves its loop as one.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* ws, int site) {
  return __all_sync(0xffffffffu, role_wait(bar, parity, abort_flag, ws, site));
}

// (The lengths and tables below are loaded from L2: the kernel before this one
// may write them while this one's CTAs are already resident.)
// Sequence b's words as loaded: loads are issued ahead and checked when they are
// needed.
struct SeqWords {
  int start, end, n;
};
__device__ __forceinline__ SeqWords seq_load(const PagedAttend& a, int b) {
  b = min(b, a.B - 1);
  return SeqWords{__ldcg(a.cu + b), __ldcg(a.cu + b + 1), __ldcg(a.kv + b)};
}
__device__ __forceinline__ bool seq_keeps(const SeqWords& w, int total, int max_q, int most) {
  return w.start >= 0 && w.end >= w.start && w.end <= total && w.end - w.start <= max_q && w.n >= 0 && w.n <= most;
}
// False (and m = 0) if the sequence breaks one of the rules that its own words show.
__device__ __forceinline__ bool seq_check(const PagedAttend& a, const SeqWords& w, SeqInfo* s) {
  const bool ok = seq_keeps(w, a.total, a.max_q, a.max_pages << a.page_shift);
  s->start = w.start;
  s->m = ok ? w.end - w.start : 0;
  s->n = w.n;
  return ok;
}

// A further rule, that a sequence's rows start where or after those of all earlier
// ones end: so no row has two sequences and the rows add up to at most `total`
// (the host's bound on the units relies on it). Where every sequence passes
// seq_check this holds by itself, since each starts where the one before ends; only
// a batch with one that does not is looked through.
// rows_before: where the rows of the sequences before b end that pass seq_check.
static __device__ __noinline__ int rows_before(const int* cu, const int* kv, int b, int total, int max_q, int most) {
  int reach = 0;
  for (int i = 0; i < b; ++i) {
    const SeqWords w{__ldcg(cu + i), __ldcg(cu + i + 1), __ldcg(kv + i)};
    if (w.end > w.start && seq_keeps(w, total, max_q, most)) reach = max(reach, w.end);
  }
  return reach;
}
__device__ __forceinline__ int rows_before(const PagedAttend& a, int b) {
  return rows_before(a.cu, a.kv, b, a.total, a.max_q, a.max_pages << a.page_shift);
}

// A CTA's run: `count` units from unit blockIdx.x * per of the line on, which is
// unit `rem` of sequence b.
template <typename U>
struct PlanRun {
  U rem;
  SeqInfo s;
  int b, count, per;
  int pairs;  // (paged_many.cu)
  U total;
  int reach;  // rows_before(b), or -1 where every sequence passes seq_check
};

// How long the runs are: an equal share, at least `least` units, and by what the
// parts take to add up; 0 (and an error) beyond any call that could end.
template <typename U>
__device__ __forceinline__ U run_length(const PagedAttend& a, int least, U total, float join) {
  const U per = max(static_cast<U>(sqrtf(join)), max(static_cast<U>(least), (total + gridDim.x - 1) / gridDim.x));
  if (per <= INT_MAX) return per;
  if (blockIdx.x == 0) raise_invalid(a.ws, 206);
  return 0;
}

// units(s): units of one key/value head of a sequence with new tokens. Runs are
// at least `least` units long (a block's, so that a tile's CTAs all have a block
// of it). U: an unsigned type that holds the call's units; the
// usual 32 bits make this half as long as 64.
// join(s): how long the parts of the sequence's largest tile take to add up, if
// cut at every unit, in units of work. A tile of b units cut into runs of x
// takes about x + join(s) / x, least at x = sqrt(join): runs are that long at
// least, so that few tiles over long texts are not cut into more parts than
// their last CTA can add up in the time the cut saves.
// Ends before the caller's next barrier; every thread of the CTA takes part.
template <int THREADS, typename U, typename Units, typename Join>
__device__ __forceinline__ void plan_run(const PagedAttend& a, int least, PlanRun<U>* run, Units units, Join join) {
  constexpr int kWarps = THREADS / 32;
  static_assert(THREADS % 32 == 0 && kWarps <= 32, "whole warps");
  __shared__ U sums[kWarps];
  __shared__ unsigned joins[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = ceil_div(a.B, THREADS);
  const int b0 = min(a.B, tid * chunk), b1 = min(a.B, b0 + chunk);
  SeqInfo s;  // of the sequence that units_of saw last
  bool good = true, ordered = true;
  auto units_of = [&](int b, bool report) -> U {
    const bool keeps = seq_check(a, seq_load(a, b), &s);
    good &= keeps;
    if (!keeps || (!ordered && s.m > 0 && s.start < rows_before(a, b))) {
      if (report && blockIdx.x == 0) raise_invalid(a.ws, -(b + 1));
      return 0;
    }
    return s.m > 0 ? units(s) * static_cast<U>(a.Hkv) : 0;
  };
  auto scan = [&](U v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const U u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  U mine, incl;
  for (;; ordered = false) {
    mine = 0;
    float longest = 0.f;
    for (int b = b0; b < b1; ++b) {
      const U u = units_of(b, true);
      mine += u;
      if (u > 0) longest = fmaxf(longest, join(s));
    }
    // (nonnegative floats order like their bits)
    const unsigned most = __reduce_max_sync(0xffffffffu, __float_as_uint(longest));
    incl = scan(mine);
    if (lane == 31) {
      sums[warp] = incl;
      joins[warp] = most;
    }
    // Once more with the further rule if some sequence is bad.
    if (__syncthreads_or(!good && ordered) == 0) break;
  }
  const U upto = scan(lane < kWarps ? sums[lane] : 0);
  const U total = __shfl_sync(0xffffffffu, upto, kWarps - 1);
  const U before = __shfl_sync(0xffffffffu, upto, warp > 0 ? warp - 1 : 0);
  const U base = (warp > 0 ? before : 0) + incl - mine;
  const float all_join = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < kWarps ? joins[lane] : 0));
  const U per = run_length<U>(a, least, total, all_join);
  const U left = per > 0 ? total : 0;
  const U first = min(left, per * blockIdx.x);
  if (tid == 0) {
    run->count = static_cast<int>(min(per, left - first));
    run->per = static_cast<int>(per);
    run->total = total;
  }
  if (first >= base && first - base < mine) {
    U rem = first - base;
    int b = b0;
    for (; chunk > 1; ++b) {  // (a thread with one sequence still holds it)
      const U u = units_of(b, false);
      if (rem < u) break;
      rem -= u;
    }
    run->b = b;
    run->reach = ordered ? -1 : rows_before(a, b);
    run->rem = rem;
    run->s = s;
  }
}

// The same for a batch of at most 32 by one warp alone, for itself: no barrier
// and one sequence per lane. Each producer warp plans so where the batch allows
// (one token over 1000 keys 8.1 -> 7.8 us; with up to four sequences per lane a
// batch of 108 took 11.8 instead of 11.1 us).
constexpr int kWarpPlan = 32;
template <typename U, typename Units, typename Join>
__device__ __forceinline__ PlanRun<U> plan_warp(const PagedAttend& a, const SeqWords& words, int least, Units units, Join join) {
  const int lane = threadIdx.x & 31;
  PlanRun<U> run;
  SeqInfo s;
  U mine = 0;
  float longest = 0.f;
  bool good = seq_check(a, words, &s);
  const bool ordered = __all_sync(0xffffffffu, good);
  int reach = -1;
  if (__builtin_expect(!ordered, 0)) {  // (rows_before by the warp)
    int upto = s.m > 0 ? s.start + s.m : 0;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) upto = max(upto, __shfl_up_sync(0xffffffffu, upto, o));
    reach = max(0, __shfl_up_sync(0xffffffffu, upto, 1));
    if (lane == 0) reach = 0;
    good &= s.m == 0 || s.start >= reach;
  }
  if (lane < a.B) {
    if (!good) {
      if (blockIdx.x == 0) raise_invalid(a.ws, -(lane + 1));
    } else if (s.m > 0) {
      mine = units(s) * static_cast<U>(a.Hkv);
      longest = join(s);
    }
  }
  U incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const U u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  const U total = __shfl_sync(0xffffffffu, incl, 31);
  const U per = run_length<U>(a, least, total, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(longest))));
  const U left = per > 0 ? total : 0, first = min(left, per * blockIdx.x);
  run.per = static_cast<int>(per);
  run.total = total;
  run.count = static_cast<int>(min(per, left - first));
  // The sequence that the run starts in.
  const U base = incl - mine;
  const unsigned who = __ballot_sync(0xffffffffu, first >= base && first - base < mine);
  run.b = who ? __ffs(who) - 1 : 0;
  run.reach = __shfl_sync(0xffffffffu, reach, run.b);
  run.rem = first - __shfl_sync(0xffffffffu, base, run.b);
  run.s = SeqInfo{__shfl_sync(0xffffffffu, s.start, run.b), __shfl_sync(0xffffffffu, s.m, run.b),
                  __shfl_sync(0xffffffffu, s.n, run.b)};
  return run;
}

// Part of one item's key blocks: blocks [j0, j1) of `blocks`. The item's first
// and last blocks lie in CTAs first_cta and last_cta, its first unit is unit
// `lead` of first_cta's run. j1 < 0 ends a run.
struct Segment {
  int start, m, n, b;
  int head, tile, j0, j1;
  int blocks, first_cta, last_cta, lead;
};
static_assert(sizeof(Segment) == 48, "three int4");

// The first block of the item that the p-th CTA after first_cta works on, with
// 2^shift units to a block.
__device__ __forceinline__ int part_begin(const Segment& s, int p, int per, int shift) {
  return p == 0 ? 0 : static_cast<int>((static_cast<long long>(p) * per - s.lead + (1 << shift) - 1) >> shift);
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
  if (!(WARP ? warp_wait(&r.full[st], ph, abort_flag, ws, site) : role_wait(&r.full[st], ph, abort_flag, ws, site)))
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
// Tiles: items(s), blocks(s, item), shift(s, item) (log2 of the units in a block)
// and before<U>(s, k) (the units of items 0 .. k - 1) of one key/value head of a
// sequence with new tokens.
// (The code is laid out so that each step of it exists once: the walk is a few
// hundred instructions that two warps run, and copies of it slowed short texts.)
template <typename U, typename Tiles>
struct RunWalker {
  const PagedAttend& a;
  const Tiles& tiles;
  const int lane, per, count;
  int reach;  // PlanRun::reach, for sequence seq_base
  int pos;    // where the current item ends, counted from the run's first unit
  Segment seg;
  SeqInfo s, next_s;
  U rem;    // before the first segment: where the run starts in its sequence
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
      bool works = x.m > 0 && seq_base + lane < a.B;
      int upto = x.m > 0 ? x.start + x.m : 0;
      if (__builtin_expect(reach >= 0, 0)) {  // a bad sequence somewhere: none may start before an earlier one's end
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) upto = max(upto, __shfl_up_sync(0xffffffffu, upto, o));
        const int before = __shfl_up_sync(0xffffffffu, upto, 1);
        works &= x.start >= (lane > 0 ? max(before, reach) : reach);
      }
      unsigned found = __ballot_sync(0xffffffffu, works);
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
      if (__builtin_expect(reach >= 0, 0)) reach = max(reach, __shfl_sync(0xffffffffu, upto, 31));
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

  __device__ __forceinline__ RunWalker(const PagedAttend& args, const Tiles& t, const PlanRun<U>& run, int ln)
      : a(args), tiles(t), lane(ln), per(run.per), count(run.count), reach(run.reach), pos(0) {
    if (count <= 0) return;
    s = run.s;
    rem = run.rem;
    seg = Segment{};
    seg.b = run.b;
    enter();
    first = entry(row, pages, 0);
    seq_base = seg.b;
    seq_cur = seq_load(a, seq_base + lane);
    seq_ahead = seq_load(a, seq_base + 32 + lane);
    next_b = -1;  // not looked for yet
  }

  // The run's first block: unit `rem` of the sequence, or the next block's start.
  __device__ __forceinline__ void find() {
    const U each = tiles.template before<U>(s, items);
    seg.head = static_cast<int>(rem / each);
    rem -= seg.head * each;
    // The last item with before(item) <= rem, 32 candidates at a time.
    for (int width = items; width > 1;) {
      const int step = (width + 31) / 32;
      const unsigned below = __ballot_sync(
          0xffffffffu, lane * step < width && tiles.template before<U>(s, seg.tile + lane * step) <= rem);
      const int l = 31 - __clz(below);
      seg.tile += l * step;
      width = min(step, width - l * step);
    }
    seg.blocks = tiles.blocks(s, seg.tile);
    const int shift = tiles.shift(s, seg.tile);
    const int off = static_cast<int>(rem - tiles.template before<U>(s, seg.tile));
    seg.j0 = (off + (1 << shift) - 1) >> shift;
    pos = ((seg.j0 < seg.blocks ? seg.j0 : seg.blocks) << shift) - off;
  }

  // On to the run's next segment (its first, at the first call); false at the end.
  __device__ __forceinline__ bool advance() {
    bool step = true;
    if (pos == 0) {  // (later on an item has ended past the run's first unit)
      if (count <= 0) return false;
      find();
      step = seg.j0 >= seg.blocks;  // the run starts inside the item's last block
    }
    if (step) {
      if (pos >= count) return false;
      seg.j0 = 0;
      if (++seg.tile == items) {
        seg.tile = 0;
        if (++seg.head == a.Hkv) {  // the next sequence
          seg.head = 0;
          if (next_b < 0) look_ahead(seg.b);
          if (next_b >= a.B) return false;
          s = next_s;
          seg.b = next_b;
          first = next_first;
          next_b = -1;
          enter();
        }
      }
      seg.blocks = tiles.blocks(s, seg.tile);
    }
    // The segment that starts at seg.j0, unit `pos` of the run. An item that began
    // before it began in the run (only a run's first can); one that does not end
    // in it is its last.
    const int me = blockIdx.x, shift = tiles.shift(s, seg.tile);
    const int len = min((count - pos + (1 << shift) - 1) >> shift, seg.blocks - seg.j0);
    const int begin = pos - (seg.j0 << shift);  // where the item begins, counted from the run's first unit
    seg.j1 = seg.j0 + len;
    seg.first_cta = seg.last_cta = me;
    seg.lead = begin;
    if (begin < 0) {
      const int back = static_cast<int>(static_cast<uint32_t>(per - 1 - begin) / static_cast<uint32_t>(per));
      seg.first_cta = me - back;
      seg.lead = back * per + begin;
    }
    if (seg.j1 < seg.blocks)
      seg.last_cta += static_cast<int>(static_cast<uint32_t>(begin + ((seg.blocks - 1) << shift)) / static_cast<uint32_t>(per));
    pos = begin + (seg.blocks << shift);  // (past the run's end where the item goes on)
    window = ((seg.j0 * kKeyBlock) >> a.page_shift) & ~31;
    cur = window == 0 ? first : entry(row, pages, window);
    ahead = entry(row, pages, window + 32);
    return true;
  }

  // After a segment's first loads: look for the sequence after this one while
  // they are on their way.
  __device__ __forceinline__ void prefetch() {
    if (next_b < 0 && pos < count) look_ahead(seg.b);
  }

  __device__ __forceinline__ int box_shift() const { return min(a.page_shift, 7); }

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

// A ring of K or of V tiles (128 keys of one head, D columns as D / 64 boxes
// columns) and the producer warp that fills it. K and V have a warp each: a lane's
// box takes about 75 cycles to issue, one after the other, and with small
// pages a block has up to 32 of them (draft tokens over 32-key pages at D = 64:
// 1400 cycles a block with one warp for both, the limit there).
template <int D>
struct TileRing {
  static constexpr int CH = D / 64, kBox = kKeyBlock * 128, kTile = CH * kBox;
  const CUtensorMap* map;
  uint8_t* tiles;
  uint64_t *full, *empty;
  uint32_t slots;
  int rb;  // keys per box: a page, or 128 of a larger one
  uint32_t st, ph, loads;

  // Load block j of the walk's segment (the whole warp).
  template <typename Walk>
  __device__ __forceinline__ bool load(Walk& walk, int j, int lane, volatile int* abort_flag, int* ws, int site) {
    const int boxes = (min(kKeyBlock, walk.seg.n - j * kKeyBlock) + rb - 1) >> walk.box_shift();  // 0 for a sequence without keys
    int row;
    const int z = walk.locate(j, lane / CH, rb, lane / CH < boxes, &row);
    if (!warp_wait(&empty[st], ph ^ 1, abort_flag, ws, site)) return false;
    if (lane == 0) mbar_arrive_expect_tx(&full[st], boxes * rb * 128 * CH);
    __syncwarp();
    if (lane < boxes * CH)
      tma_load_3d(tiles + st * kTile + (lane % CH) * kBox + (lane / CH) * rb * 128, map, &full[st], (lane % CH) * 64, row,
                  z);
    __syncwarp();
    ++loads;
    if (++st == slots) { st = 0; ph ^= 1; }
    return true;
  }

  // An aborting producer lets its copies in flight land before the CTA exits.
  __device__ __forceinline__ void settle() const {
    int never = 0;
    for (uint32_t s = 0; s < slots && s < loads; ++s) {
      const uint32_t idx = loads - 1 - s;
      mbar_wait(&full[idx % slots], (idx / slots) & 1, &never, nullptr, 0);
    }
  }
};

// The count of a cut tile's stored parts is one byte in the workspace header, put
// back to zero by whoever finds it complete.
struct PartCount {
  int* word;
  int shift, parts;

  __device__ __forceinline__ PartCount(const Segment& seg, int* ws)
      : word(ws + kHdrParts + (seg.first_cta >> 2)), shift(8 * (seg.first_cta & 3)), parts(seg.last_cta - seg.first_cta + 1) {}

  // Counts this CTA's part (whose stores happened before, by a barrier): was it
  // the last? Released, so that whoever sees this count sees the part, and
  // acquired, so that whoever is last sees the others' (one instruction: with
  // fences around a plain atomic this took 3500 cycles).
  __device__ __forceinline__ bool add() const {
    unsigned before;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(before) : "l"(word), "r"(1u << shift) : "memory");
    const bool last = ((before >> shift) & 255u) == static_cast<unsigned>(parts - 1);
    if (last) clear(parts);
    return last;
  }

  // Are the other CTAs' parts all there (and visible)? If so this CTA need not
  // store its own.
  __device__ __forceinline__ bool others() const {
    unsigned now;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(word) : "memory");
    const bool all = ((now >> shift) & 255u) == static_cast<unsigned>(parts - 1);
    if (all) clear(parts - 1);
    return all;
  }

  __device__ __forceinline__ void clear(int n) const {
    atomicSub(reinterpret_cast<unsigned*>(word), static_cast<unsigned>(n) << shift);
  }
};

// (out of line: two calls)
static __device__ __noinline__ bool part_count(const Segment& seg, int* ws) { return PartCount(seg, ws).add(); }

// After every epilogue warp of this CTA has stored its share of a tile's
// part: *last_flag tells whether this CTA's part was the tile's last (uniform over
// the CTA's epilogue warps; the other parts are then visible). `ph`: parity of
// the two barriers, flipped by the caller each time.
__device__ __forceinline__ bool last_part(uint64_t* stored, uint64_t* counted, int* last_flag, const Segment& seg,
                                          int* ws, int warp, int lane, uint32_t ph, volatile int* abort_flag, int site) {
  // (The barrier orders every warp's stores before the count.)
  __syncwarp();
  if (lane == 0) mbar_arrive(stored);
  if (warp == 0) {
    if (!warp_wait(stored, ph, abort_flag, ws, site)) return false;
    if (lane == 0) {
      *last_flag = part_count(seg, ws);
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
