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
#pragma once

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
__device__ __forceinline__ bool seq_info(const PagedAttend& a, int b, SeqInfo* s) {
  const int start = __ldcg(a.cu + b), end = __ldcg(a.cu + b + 1), n = __ldcg(a.kv + b);
  const bool ok = start >= 0 && end >= start && end <= a.total && end - start <= a.max_q && n >= 0 &&
                  n <= a.max_pages << a.page_shift;
  s->start = start;
  s->m = ok ? end - start : 0;
  s->n = n;
  return ok;
}

// A CTA's run: units [first, first + count), `per` units to a CTA; its first
// unit is unit `rem` of sequence b.
struct PlanRun {
  long long first, count, per, rem;
  int b;
};

// units(s): units of one key/value head of a sequence with new tokens. Runs are
// at least a.least units long (a run's fixed costs are then worth paying).
// Ends before the caller's next barrier; every thread of the CTA takes part.
template <int THREADS, typename Units>
__device__ __forceinline__ void plan_run(const PagedAttend& a, PlanRun* run, Units units) {
  static_assert(THREADS % 32 == 0, "whole warps");
  __shared__ long long sums[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = ceil_div(a.B, THREADS);
  const int b0 = min(a.B, tid * chunk), b1 = min(a.B, b0 + chunk);
  auto units_of = [&](int b, bool report) -> long long {
    SeqInfo s;
    if (!seq_info(a, b, &s)) {
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
  const long long per = max(static_cast<long long>(a.least), (total + gridDim.x - 1) / gridDim.x);
  const long long first = min(total, per * blockIdx.x);
  if (tid == 0) {
    run->first = first;
    run->count = min(per, total - first);
    run->per = per;
  }
  if (first >= base && first < base + mine) {
    long long rem = first - base;
    int b = b0;
    for (;; ++b) {
      const long long u = units_of(b, false);
      if (rem < u) break;
      rem -= u;
    }
    run->b = b;
    run->rem = rem;
  }
}

// Part of one tile's key blocks: blocks [j0, j1) of `blocks`; the tile's
// first and last blocks lie in CTAs first_cta and last_cta. j1 < 0 ends a run.
struct Segment {
  int start, m, n, b;
  int head, tile, j0, j1;
  int blocks, first_cta, last_cta;
  int lead;  // the first CTA's units before the tile (a part p CTAs on starts at block p * per - lead)
};
static_assert(sizeof(Segment) == 48, "three int4");

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

// The page numbers of the blocks a producer warp is about to load: lane l holds
// table entry base + l, and the next 32 are on the way.
struct PageWindow {
  const int* row;
  int base, pages, cur, next;
  __device__ __forceinline__ int entry(int i, int lane) const { return i + lane < pages ? __ldcg(row + i + lane) : -1; }
  __device__ __forceinline__ PageWindow(const PagedAttend& a, int b, int n, int key0, int lane)
      : row(a.table + static_cast<size_t>(b) * a.max_pages), base(key0 >> a.page_shift),
        pages((n + (1 << a.page_shift) - 1) >> a.page_shift) {
    cur = entry(base, lane);
    next = entry(base + 32, lane);
  }
  // Where box `box` (of rb keys) of the block at key0 lies: the slice (page *
  // Hkv + head) and *r, the row in it. A bad page (reported where `used`)
  // lies past the last slice, where a load reads zeros. Blocks come in order.
  __device__ __forceinline__ int locate(const PagedAttend& a, int key0, int box, int rb, bool used, int head, int* r) {
    if ((key0 >> a.page_shift) >= base + 32) {
      base += 32;
      cur = next;
      next = entry(base + 32, threadIdx.x & 31);
    }
    const int key = key0 + box * rb;
    const int page = __shfl_sync(0xffffffffu, cur, ((key >> a.page_shift) - base) & 31);
    *r = key & ((1 << a.page_shift) - 1);
    if (page >= 0 && page < a.num_pages) return page * a.Hkv + head;
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
  __threadfence();
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
