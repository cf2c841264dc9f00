// pages.cu -- the paged cache's bookkeeping: taking pages for new tokens
// (sigattn_paged_reserve) and giving pages back (sigattn_paged_release); and its
// writer (sigattn_paged_write).
//
// The bookkeeping turns per-sequence lengths into per-token and per-page work with
// prefix sums over the batch (B <= 4096). Every CTA forms the whole sums itself
// from the lengths (8 bytes per sequence, from L2), so one launch does the call and
// no CTA waits for another; the CTAs then share the tokens and pages out. Words
// that a caller may pass as input and output at once (the stack height, the
// lengths) are written by the CTA that came last to have read them.
// Latency bounds both calls (a few thousand bytes): what counts is the chain
// lengths -> sums -> pages -> slots, one trip to memory each.
#include "paged.cuh"

namespace sigattn {

namespace {

constexpr int kThreads = 256;

// Exclusive prefix sums over the CTA of a pair of values per thread; the totals go
// to *total_x, *total_y of every thread.
__device__ __forceinline__ void block_scan2(uint32_t& x, uint32_t& y, uint32_t* total_x, uint32_t* total_y) {
  constexpr int kWarps = kThreads / 32;
  __shared__ uint2 sums[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](uint2 v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t ux = __shfl_up_sync(0xffffffffu, v.x, o), uy = __shfl_up_sync(0xffffffffu, v.y, o);
      if (lane >= o) {
        v.x += ux;
        v.y += uy;
      }
    }
    return v;
  };
  const uint2 incl = scan(make_uint2(x, y));
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  const uint2 upto = scan(lane < kWarps ? sums[lane] : make_uint2(0, 0));
  *total_x = __shfl_sync(0xffffffffu, upto.x, kWarps - 1);
  *total_y = __shfl_sync(0xffffffffu, upto.y, kWarps - 1);
  const uint32_t bx = __shfl_sync(0xffffffffu, upto.x, warp > 0 ? warp - 1 : 0);
  const uint32_t by = __shfl_sync(0xffffffffu, upto.y, warp > 0 ? warp - 1 : 0);
  x = (warp > 0 ? bx : 0) + incl.x - x;
  y = (warp > 0 ? by : 0) + incl.y - y;
}

// The last b with off[b] <= i, for off[0] = 0 <= i < off[B] (so sequence b
// owns element i, empty sequences skipped).
__device__ __forceinline__ int owner(const int* off, int B, int i) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Pages of n tokens.
__device__ __forceinline__ int pages_of(int n, int shift) { return (n + (1 << shift) - 1) >> shift; }

// Thread 0 of a CTA that has read all it needs of the lengths and the height:
// whether it is the grid's last (the ticket word is then back at zero).
__device__ __forceinline__ bool last_reader(int* ws) {
  if (gridDim.x == 1) return true;
  if (atomicAdd(ws + kHdrTicket, 1) != static_cast<int>(gridDim.x) - 1) return false;
  ws[kHdrTicket] = 0;
  return true;
}

}  // namespace

// AHEAD: a call of one CTA and of no more sequences than threads. The pages that the
// sequences go on in and the stack's top are then loaded while the sums are
// formed: 64 single tokens 4.1 -> 3.6 us. (In larger calls and for released pages it
// is no gain: 256 prompts 5.7 -> 5.9 us, tails of 64 sequences 3.3 either way.)
template <bool AHEAD>
__global__ void __launch_bounds__(kThreads) reserve_kernel(PagedReserve a) {
  grid_dep_launch();
  grid_dep_wait();
  extern __shared__ int smem_pages[];
  __shared__ int s_bad, s_last, s_count;
  __shared__ float s_tokens;
  int* s_cached = smem_pages;          // [B] tokens before the call
  int* s_cu = s_cached + a.B;          // [B + 1] new tokens before sequence b
  int* s_pg = s_cu + a.B + 1;          // [B + 1] new pages before sequence b
  __shared__ int s_page[AHEAD ? kThreads : 1];   // the page that sequence b goes on in
  __shared__ int s_stack[AHEAD ? kThreads : 1];  // the stack's top pages
  const int tid = threadIdx.x;
  const int sh = a.page_shift, ps = 1 << sh;
  const int most = a.max_pages << sh;
  if (tid == 0) {
    s_bad = a.B;
    s_tokens = 0.f;
    s_count = *a.free_count;  // read by one thread, so that its CTA has read it where it says so
  }
  const int per = ceil_div(a.B, kThreads);
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  uint32_t tok = 0, pg = 0;
  float tokens = 0.f;  // so many that 32 bits would not hold them show here
  int worst = a.B;
  int page0 = -1, top = -1;
  for (int b = b0; b < b1; ++b) {
    const int c = a.cached[b], m = a.fresh[b];
    s_cached[b] = c;
    s_cu[b] = m;
    if (c < 0 || m < 0 || c > most || m > most - c || m > a.max_new) {
      worst = min(worst, b);
    } else {
      tok += m;
      tokens += m;
      pg += pages_of(c + m, sh) - pages_of(c, sh);
      if (AHEAD && m > 0 && (c & (ps - 1)) != 0) page0 = a.table[static_cast<size_t>(b) * a.max_pages + (c >> sh)];
    }
  }
  __syncthreads();
  if (AHEAD && s_count <= a.num_pages && tid < s_count) top = a.free_pages[s_count - 1 - tid];
  if (worst < a.B) atomicMin(&s_bad, worst);
  if (tokens > 1e6f) atomicAdd(&s_tokens, tokens);
  uint32_t total_tok, total_pg;
  block_scan2(tok, pg, &total_tok, &total_pg);  // its barrier also covers s_bad and s_tokens
  // Every thread of the CTA has its lengths and the height.
  if (tid == 0) s_last = last_reader(a.ws);
  const int bad = s_bad, count = s_count;
  const bool many = s_tokens > 2e9f || total_tok > static_cast<uint32_t>(a.rows);
  const bool few = count < 0 || count > a.num_pages || total_pg > static_cast<uint32_t>(count);
  const bool ok = bad == a.B && !many && !few;
  if (!ok && blockIdx.x == 0 && tid == 0) raise_invalid(a.ws, bad < a.B ? -(bad + 1) : many ? 201 : 202);
  for (int b = b0; b < b1; ++b) {
    const int c = s_cached[b], m = ok ? s_cu[b] : 0;
    s_cu[b] = ok ? static_cast<int>(tok) : 0;
    s_pg[b] = ok ? static_cast<int>(pg) : 0;
    tok += m;
    pg += pages_of(c + m, sh) - pages_of(c, sh);
  }
  const int T = ok ? static_cast<int>(total_tok) : 0, P = ok ? static_cast<int>(total_pg) : 0;
  if (tid == 0) {
    s_cu[a.B] = T;
    s_pg[a.B] = P;
  }
  if (AHEAD) {
    s_page[tid] = page0;
    s_stack[tid] = top;
  }
  __syncthreads();
  if (s_last) {
    for (int b = tid; b <= a.B; b += kThreads) {
      a.cu[b] = s_cu[b];
      if (b < a.B) a.kv[b] = s_cached[b] + s_cu[b + 1] - s_cu[b];
    }
    if (tid == 0) *a.free_count_out = count - P;
  }

  // Slots and positions, four consecutive rows per thread and step: one search
  // for the first, the others by counting on. New page i (in batch order) is
  // stack[count - 1 - i]; it starts with a new token, whose thread enters it in
  // the table. Pages past the ones in use come from the stack, so no CTA reads
  // what another one wrote.
  const bool wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
  const int groups = a.rows / 4 + (a.rows % 4 != 0);
  for (int g = blockIdx.x * kThreads + tid; g < groups; g += gridDim.x * kThreads) {
    const int t0 = 4 * g;
    int slot[4] = {-1, -1, -1, -1}, at[4] = {0, 0, 0, 0};
    if (t0 < T) {
      int b = owner(s_cu, a.B, t0);
      int c = s_cached[b], have = pages_of(c, sh), seen = -1, page = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t0 + e;
        if (t >= T) break;
        if (t >= s_cu[b + 1]) {
          do ++b; while (t >= s_cu[b + 1]);
          c = s_cached[b];
          have = pages_of(c, sh);
          seen = -1;
        }
        at[e] = c + t - s_cu[b];
        const int k = at[e] >> sh;
        if (k != seen) {
          seen = k;
          int* entry = a.table + static_cast<size_t>(b) * a.max_pages + k;
          const int i = s_pg[b] + k - have;  // which new page
          if (AHEAD && (k < have || i < kThreads))
            page = k < have ? s_page[b] : s_stack[i];
          else
            page = k < have ? *entry : a.free_pages[count - 1 - i];
          if (page < 0 || page >= a.num_pages) {
            raise_invalid(a.ws, 203);
            page = -1;
          }
          if (k >= have && (at[e] & (ps - 1)) == 0) *entry = page;
        }
        if (page >= 0) slot[e] = (page << sh) + (at[e] & (ps - 1));
      }
    }
    if (wide && t0 + 4 <= a.rows) {
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (a.positions) *reinterpret_cast<int4*>(a.positions + t0) = make_int4(at[0], at[1], at[2], at[3]);
    } else {
      for (int e = 0; e < 4 && t0 + e < a.rows; ++e) {
        a.slots[t0 + e] = slot[e];
        if (a.positions) a.positions[t0 + e] = at[e];
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads) release_kernel(PagedRelease a) {
  grid_dep_launch();
  grid_dep_wait();
  extern __shared__ int smem_pages[];
  __shared__ int s_bad, s_last, s_count;
  __shared__ float s_pages;
  int* s_pg = smem_pages;           // [B + 1] released pages before sequence b
  int* s_first = s_pg + a.B + 1;    // [B] the first page it gives back
  const int tid = threadIdx.x;
  const int sh = a.page_shift;
  const int most = a.max_pages << sh;
  if (tid == 0) {
    s_bad = a.B;
    s_pages = 0.f;
    s_count = *a.free_count;
  }
  const int per = ceil_div(a.B, kThreads);
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  uint32_t pg = 0, unused = 0, total, total_unused;
  float pages = 0.f;
  int worst = a.B;
  for (int b = b0; b < b1; ++b) {
    const int n = a.kv[b], keep = a.keep ? a.keep[b] : 0;
    const bool bad = keep < 0 || n < keep || n > most;
    const int gone = bad ? 0 : pages_of(n, sh) - pages_of(keep, sh);
    if (bad) worst = min(worst, b);
    s_first[b] = bad ? 0 : pages_of(keep, sh);
    s_pg[b] = gone;
    pg += gone;
    pages += gone;
  }
  __syncthreads();
  if (worst < a.B) atomicMin(&s_bad, worst);
  if (pages > 1e6f) atomicAdd(&s_pages, pages);
  block_scan2(pg, unused, &total, &total_unused);
  const int bad = s_bad, count = s_count;
  const bool fits = count >= 0 && count <= a.num_pages && s_pages < 2e9f &&
                    total <= static_cast<uint32_t>(a.num_pages - count);
  const bool ok = bad == a.B && fits;
  const int P = ok ? static_cast<int>(total) : 0;
  if (tid == 0) {
    if (!ok && blockIdx.x == 0) raise_invalid(a.ws, bad < a.B ? -(bad + 1) : 202);
    s_last = last_reader(a.ws);
    if (s_last) *a.free_count_out = count + P;
    s_pg[a.B] = P;
  }
  for (int b = b0; b < b1; ++b) {
    const int gone = s_pg[b];
    s_pg[b] = static_cast<int>(pg);
    pg += gone;
  }
  __syncthreads();
  if (s_last && a.kv_out != nullptr)
    for (int b = tid; b < a.B; b += kThreads) a.kv_out[b] = !ok ? a.kv[b] : a.keep ? a.keep[b] : 0;
  for (int i = blockIdx.x * kThreads + tid; i < P; i += gridDim.x * kThreads) {
    const int b = owner(s_pg, a.B, i);
    int page = a.table[static_cast<size_t>(b) * a.max_pages + s_first[b] + i - s_pg[b]];
    if (page < 0 || page >= a.num_pages) {
      raise_invalid(a.ws, 203);
      page = -1;
    }
    a.free_pages[count + i] = page;
  }
}

namespace {

// The lengths and sums of the largest batches take more than 48 KB.
constexpr int kPagesSmem = (3 * kMaxBatch + 2) * static_cast<int>(sizeof(int));

cudaError_t pages_setup() {
  static PerDeviceOnce attr;
  return attr.run([] {
    const cudaError_t e = cudaFuncSetAttribute(reserve_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPagesSmem);
    return e != cudaSuccess ? e
                            : cudaFuncSetAttribute(release_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPagesSmem);
  });
}

}  // namespace

cudaError_t launch_paged_reserve(const PagedReserve& a, int num_sms, cudaStream_t stream) {
  const cudaError_t e = pages_setup();
  if (e != cudaSuccess) return e;
  const int smem = (3 * a.B + 2) * static_cast<int>(sizeof(int));
  const long long work = static_cast<long long>(a.rows) / 4 + 1;
  const int grid = static_cast<int>(std::max<long long>(1, std::min<long long>(2 * num_sms, (work + kThreads - 1) / kThreads)));
  return launch_programmatic(grid == 1 && a.B <= kThreads ? reserve_kernel<true> : reserve_kernel<false>, dim3(grid),
                             dim3(kThreads), smem, stream, a);
}

cudaError_t launch_paged_release(const PagedRelease& a, int num_sms, cudaStream_t stream) {
  const cudaError_t e = pages_setup();
  if (e != cudaSuccess) return e;
  const int smem = (2 * a.B + 1) * static_cast<int>(sizeof(int));
  const long long work = static_cast<long long>(a.B) * a.max_pages;
  const int grid =
      static_cast<int>(std::max<long long>(1, std::min<long long>(2 * num_sms, (work + 4 * kThreads - 1) / (4 * kThreads))));
  return launch_programmatic(release_kernel, dim3(grid), dim3(kThreads), smem, stream, a);
}

// ---------------------------------------------------------------------------
// Cache writes with rotary positions
// ---------------------------------------------------------------------------
// A warp takes one token, or (few tokens) a share of one token's heads. A lane's
// unit is 16 values of a head, two 16-byte chunks, the same two for every
// head, so its cosines and sines stay in registers over all heads. With halves
// the unit holds both members of eight pairs (chunks c and c + pairs / 8): it
// reads all it needs before it writes, and q_out may be q itself. The warp
// starts its first heads' loads, then its lanes form the token's cosines and
// sines once (the angle in 64 bits, as turns, so its reduction is a
// subtraction; sincospif of the remainder) and pass them on through shared
// memory. With more tokens than warps a warp goes from token to token, the next
// rows, slots and positions on their way meanwhile. Bound by reading and writing
// the rows: 16384 tokens of 48 heads of 128 take 66 us, 93 % of the copy rate (a CTA
// per token, with a barrier between its angles and its rows: 140 us; a warp per
// token without the loop: 69 us, and 18 instead of 12 us where a token has 6 heads
// of 64). Three steps of rows ahead at 16 warps per SM: two 70 us, four 72 us.
constexpr int kWriteWarps = 4;

template <bool ADJACENT>
__global__ void __launch_bounds__(kWriteWarps * 32, 4) write_kernel(PagedWrite a) {
  grid_dep_launch();
  grid_dep_wait();
  __shared__ float2 s_turn[kWriteWarps][64];
  const int lane = threadIdx.x & 31;
  const int lanes = a.d / 16, abreast = 32 / lanes;  // lanes per head, heads at once
  const int l = lane % lanes, sub = lane / lanes;
  const int heads = a.Hq + 2 * a.Hkv, steps = (heads + abreast - 1) / abreast;
  // The warp's tokens and its share of their heads.
  const int warps = gridDim.x * kWriteWarps / a.shares;  // tokens at once
  const int unit = blockIdx.x * kWriteWarps + (threadIdx.x >> 5);
  const int share = unit % a.shares;
  const int first = share * steps / a.shares, last = (share + 1) * steps / a.shares;
  const int pc = a.pairs / 8;  // chunks of the first members (halves)
  // The lane's chunks of a turned head, and whether they turn.
  int c0 = 2 * l, c1 = 2 * l + 1;
  bool turns = false;
  if (ADJACENT) {
    turns = c0 * 4 < a.pairs;
  } else if (l < pc) {
    c0 = l;
    c1 = l + pc;
    turns = true;
  }

  struct Row {
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;  // null: nothing to do
    bool v;
  };
  auto row_of = [&](long long t, int slot, int step) {
    const int head = step * abreast + sub;
    const bool stored = slot >= 0 && (slot >> a.page_shift) < a.num_pages;
    Row r{nullptr, nullptr, false};
    if (head < a.Hq) {
      r.src = a.q + t * a.q_stride + head * a.d;
      r.dst = a.q_out + t * a.q_out_stride + head * a.d;
    } else if (head < heads && stored) {
      r.v = head >= a.Hq + a.Hkv;
      const int h = head - a.Hq - (r.v ? a.Hkv : 0);
      r.src = r.v ? a.v + t * a.v_stride + h * a.d : a.k + t * a.k_stride + h * a.d;
      r.dst = (r.v ? a.v_cache : a.k_cache) +
              (((static_cast<size_t>(slot >> a.page_shift) * a.Hkv + h) << a.page_shift) + (slot & ((1 << a.page_shift) - 1))) *
                  a.d;
    }
    return r;
  };
  // (a value row is copied by the lane's own two chunks in order)
  auto fetch = [&](const Row& r, uint4& x, uint4& y) {
    if (r.dst == nullptr) return;
    const uint4* src = reinterpret_cast<const uint4*>(r.src);
    x = src[r.v ? 2 * l : c0];
    y = src[r.v ? 2 * l + 1 : c1];
  };
  // The positions of the lane's pairs lane and lane + 32, as 64-bit floats.
  int axis[2] = {0, 0};
  double freq[2] = {0.0, 0.0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int p = lane + 32 * i;
    if (p >= a.pairs) continue;
    freq[i] = static_cast<double>(a.inv_freq[p]) * 0.15915494309189535;  // 1 / (2 pi): angles in turns
    axis[i] = a.pair_axis ? a.pair_axis[p] : 0;
    if (axis[i] < 0 || axis[i] >= a.axes) {
      raise_invalid(a.ws, 205);
      axis[i] = 0;
    }
  }
  auto position = [&](long long t, int i) {
    return lane + 32 * i < a.pairs ? a.positions[static_cast<long long>(axis[i]) * a.rows + t] : 0;
  };

  long long t = unit / a.shares;
  if (t >= a.rows) return;
  float2* turn = s_turn[threadIdx.x >> 5];
  constexpr int kAhead = 3;
  uint4 x[kAhead], y[kAhead];
  int slot = a.slots[t];
  int pos[2] = {position(t, 0), position(t, 1)};
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (first + i < last) fetch(row_of(t, slot, first + i), x[i], y[i]);
  for (; t < a.rows; t += warps) {
    const long long tn = t + warps;
    const bool more = tn < a.rows;
    const int next_slot = more ? a.slots[tn] : -1;
    if ((slot < -1 || (slot >= 0 && (slot >> a.page_shift) >= a.num_pages))) raise_invalid(a.ws, 204);
    // This token's cosines and sines.
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = lane + 32 * i;
      if (p < a.pairs) {
        const double angle = pos[i] * freq[i];
        float sn, cn;
        sincospif(2.0f * static_cast<float>(angle - rint(angle)), &sn, &cn);
        turn[p] = make_float2(cn, sn);
      }
      if (more) pos[i] = position(tn, i);
    }
    __syncwarp();
    float2 cs[8];  // of the lane's pairs
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int p = ADJACENT ? c0 * 4 + e : c0 * 8 + e;
      cs[e] = turns && p < a.pairs ? turn[p] : make_float2(1.0f, 0.0f);
    }
    auto finish = [&](const Row& r, const uint4& xx, const uint4& yy) {
      if (r.dst == nullptr) return;
      uint32_t xw[4] = {xx.x, xx.y, xx.z, xx.w}, yw[4] = {yy.x, yy.y, yy.z, yy.w};
      uint4* dst = reinterpret_cast<uint4*>(r.dst);
      if (turns && !r.v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (ADJACENT) {
            xw[e] = turn_word(xw[e], cs[e]);
            if (c1 * 4 < a.pairs) yw[e] = turn_word(yw[e], cs[4 + e]);
          } else {
            turn_words(xw[e], yw[e], cs[2 * e], cs[2 * e + 1]);
          }
        }
      }
      dst[r.v ? 2 * l : c0] = make_uint4(xw[0], xw[1], xw[2], xw[3]);
      dst[r.v ? 2 * l + 1 : c1] = make_uint4(yw[0], yw[1], yw[2], yw[3]);
    };
    for (int s0 = first; s0 < last; s0 += kAhead) {
      uint4 nx[kAhead], ny[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        nx[i] = x[i];
        ny[i] = y[i];
      }
      // The next rows: of this token, or the first of the next one.
      const bool here = s0 + kAhead < last;
      const int sn = here ? s0 + kAhead : first;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if ((here || more) && sn + i < last) fetch(row_of(here ? t : tn, here ? slot : next_slot, sn + i), x[i], y[i]);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (s0 + i < last) finish(row_of(t, slot, s0 + i), nx[i], ny[i]);
    }
    slot = next_slot;
  }
}

cudaError_t launch_paged_write(PagedWrite a, int num_sms, cudaStream_t stream) {
  const int abreast = 32 / (a.d / 16);
  const int steps = (a.Hq + 2 * a.Hkv + abreast - 1) / abreast;
  // A token's heads are shared out until the GPU has 16 warps per SM; with more
  // tokens than that, warps go from token to token.
  a.shares = static_cast<int>(std::max<long long>(1, std::min<long long>(steps, 16LL * num_sms / a.rows)));
  const long long units = static_cast<long long>(a.rows) * a.shares;
  const long long ctas = std::min<long long>(4LL * num_sms, (units + kWriteWarps - 1) / kWriteWarps);
  // whole tokens at once: the warps are a multiple of the shares
  const int grid = static_cast<int>((ctas + a.shares - 1) / a.shares * a.shares);
  return launch_programmatic(a.adjacent ? write_kernel<true> : write_kernel<false>, dim3(grid), dim3(kWriteWarps * 32),
                             0, stream, a);
}

}  // namespace sigattn
