// pages.cu -- the paged cache's bookkeeping: taking pages for new tokens
// (sigattn_paged_reserve) and giving pages back (sigattn_paged_release).
//
// Both turn per-sequence lengths into per-token and per-page work with prefix
// sums over the batch (B <= 4096). Every CTA forms the whole sums itself from
// the lengths (16 bytes per sequence, from L2), so one launch does the call and
// no CTA waits for another; the CTAs then share the tokens and pages out. Words
// that a caller may pass as input and output at once (the stack height, the
// lengths) are written by the CTA that finishes last, when every CTA has read
// them.
#include "paged.cuh"

namespace sigattn {

namespace {

constexpr int kThreads = 256;

// Exclusive prefix sums over the CTA of one pair of 64-bit values per thread
// (64 bits: a batch of bad lengths may add up to more than 32); the totals
// go to *total_x, *total_y of every thread.
__device__ __forceinline__ void block_scan2(long long& x, long long& y, long long* total_x, long long* total_y) {
  __shared__ long long sums[2][kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ix = x, iy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ux = __shfl_up_sync(0xffffffffu, ix, o), uy = __shfl_up_sync(0xffffffffu, iy, o);
    if (lane >= o) {
      ix += ux;
      iy += uy;
    }
  }
  if (lane == 31) {
    sums[0][warp] = ix;
    sums[1][warp] = iy;
  }
  __syncthreads();
  long long bx = 0, by = 0, tx = 0, ty = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) {
      bx = tx;
      by = ty;
    }
    tx += sums[0][w];
    ty += sums[1][w];
  }
  x = bx + ix - x;
  y = by + iy - y;
  *total_x = tx;
  *total_y = ty;
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

// Whether this CTA is the last of the grid to come here (uniform over the
// CTA); the header's ticket word is back at zero afterwards. What every other
// CTA read or wrote before is ordered before what the last one does next.
__device__ __forceinline__ bool last_cta(int* ws) {
  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = gridDim.x == 1 || atomicAdd(ws + kHdrTicket, 1) == static_cast<int>(gridDim.x) - 1;
    if (last) ws[kHdrTicket] = 0;
    __threadfence();
  }
  __syncthreads();
  return last != 0;
}

}  // namespace

__global__ void __launch_bounds__(kThreads) reserve_kernel(PagedReserve a) {
  grid_dep_launch();
  grid_dep_wait();
  extern __shared__ int smem_pages[];
  __shared__ int s_bad;
  int* s_cu = smem_pages;                // [B + 1] new tokens before sequence b
  int* s_pg = smem_pages + a.B + 1;      // [B + 1] new pages before sequence b
  const int tid = threadIdx.x;
  const int sh = a.page_shift, ps = 1 << sh;
  const int most = a.max_pages << sh;
  if (tid == 0) s_bad = a.B;
  __syncthreads();
  const int per = ceil_div(a.B, kThreads);
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  const int count = *a.free_count;
  long long tok = 0, pg = 0;
  for (int b = b0; b < b1; ++b) {
    const int c = a.cached[b], m = a.fresh[b];
    if (c < 0 || m < 0 || c > most || m > most - c) {
      atomicMin(&s_bad, b);
    } else {
      tok += m;
      pg += ((c + m + ps - 1) >> sh) - ((c + ps - 1) >> sh);
    }
  }
  long long total_tok, total_pg;
  block_scan2(tok, pg, &total_tok, &total_pg);  // its barrier also covers s_bad
  const int bad = s_bad;
  const bool few = count < 0 || count > a.num_pages || total_pg > count;
  const bool ok = bad == a.B && total_tok <= a.rows && !few;
  if (!ok && blockIdx.x == 0 && tid == 0)
    raise_invalid(a.ws, bad < a.B ? -(bad + 1) : total_tok > a.rows ? 201 : 202);
  if (ok) {
    for (int b = b0; b < b1; ++b) {
      const int c = a.cached[b], m = a.fresh[b];
      s_cu[b] = static_cast<int>(tok);
      s_pg[b] = static_cast<int>(pg);
      tok += m;
      pg += ((c + m + ps - 1) >> sh) - ((c + ps - 1) >> sh);
    }
  }
  const int T = ok ? static_cast<int>(total_tok) : 0, P = ok ? static_cast<int>(total_pg) : 0;
  if (tid == 0) {
    s_cu[a.B] = T;
    s_pg[a.B] = P;
  }
  __syncthreads();
  const int gid = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;

  // New table entries: new page i (in batch order) is stack[count - 1 - i].
  for (int i = gid; i < P; i += gsize) {
    const int b = owner(s_pg, a.B, i);
    const int k = ((a.cached[b] + ps - 1) >> sh) + i - s_pg[b];
    int page = a.free_pages[count - 1 - i];
    if (page < 0 || page >= a.num_pages) {
      raise_invalid(a.ws, 203);
      page = -1;
    }
    a.table[static_cast<size_t>(b) * a.max_pages + k] = page;
  }
  // Slots and positions, four consecutive rows per thread and step: one search
  // for the first, the others by counting on. Pages of new tokens past the
  // ones in use come from the stack, so no CTA reads what another one wrote.
  const bool wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
  const int groups = a.rows / 4 + (a.rows % 4 != 0);
  for (int g = gid; g < groups; g += gsize) {
    const int t0 = 4 * g;
    int slot[4] = {-1, -1, -1, -1}, at[4] = {0, 0, 0, 0};
    if (t0 < T) {
      int b = owner(s_cu, a.B, t0);
      int c = a.cached[b], have = (c + ps - 1) >> sh, seen = -1, page = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t0 + e;
        if (t >= T) break;
        if (t >= s_cu[b + 1]) {
          do ++b; while (t >= s_cu[b + 1]);
          c = a.cached[b];
          have = (c + ps - 1) >> sh;
          seen = -1;
        }
        at[e] = c + t - s_cu[b];
        const int k = at[e] >> sh;
        if (k != seen) {
          seen = k;
          page = k < have ? a.table[static_cast<size_t>(b) * a.max_pages + k]
                          : a.free_pages[count - 1 - (s_pg[b] + k - have)];
          if (page < 0 || page >= a.num_pages) {
            raise_invalid(a.ws, 203);
            page = -1;
          }
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

  if (!last_cta(a.ws)) return;
  for (int b = tid; b <= a.B; b += kThreads) {
    a.cu[b] = ok ? s_cu[b] : 0;
    if (b < a.B) a.kv[b] = a.cached[b] + (ok ? s_cu[b + 1] - s_cu[b] : 0);
  }
  if (tid == 0) *a.free_count_out = count - P;
}

__global__ void __launch_bounds__(kThreads) release_kernel(PagedRelease a) {
  grid_dep_launch();
  grid_dep_wait();
  extern __shared__ int smem_pages[];
  __shared__ int s_bad;
  int* s_pg = smem_pages;  // [B + 1] released pages before sequence b
  const int tid = threadIdx.x;
  const int sh = a.page_shift, ps = 1 << sh;
  const int most = a.max_pages << sh;
  if (tid == 0) s_bad = a.B;
  __syncthreads();
  const int per = ceil_div(a.B, kThreads);
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  const int count = *a.free_count;
  long long pg = 0, unused = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = a.kv[b], keep = a.keep ? a.keep[b] : 0;
    if (keep < 0 || n < keep || n > most) atomicMin(&s_bad, b);
    else pg += ((n + ps - 1) >> sh) - ((keep + ps - 1) >> sh);
  }
  long long total, total_unused;
  block_scan2(pg, unused, &total, &total_unused);
  const int bad = s_bad;
  const bool ok = bad == a.B && count >= 0 && total <= a.num_pages - count;
  if (!ok && blockIdx.x == 0 && tid == 0) raise_invalid(a.ws, bad < a.B ? -(bad + 1) : 202);
  if (ok) {
    for (int b = b0; b < b1; ++b) {
      const int n = a.kv[b], keep = a.keep ? a.keep[b] : 0;
      s_pg[b] = static_cast<int>(pg);
      pg += ((n + ps - 1) >> sh) - ((keep + ps - 1) >> sh);
    }
  }
  const int P = ok ? static_cast<int>(total) : 0;
  if (tid == 0) s_pg[a.B] = P;
  __syncthreads();
  for (int i = blockIdx.x * kThreads + tid; i < P; i += gridDim.x * kThreads) {
    const int b = owner(s_pg, a.B, i);
    const int keep = a.keep ? a.keep[b] : 0;
    int page = a.table[static_cast<size_t>(b) * a.max_pages + ((keep + ps - 1) >> sh) + i - s_pg[b]];
    if (page < 0 || page >= a.num_pages) {
      raise_invalid(a.ws, 203);
      page = -1;
    }
    a.free_pages[count + i] = page;
  }
  if (last_cta(a.ws) && tid == 0) *a.free_count_out = count + P;
}

cudaError_t launch_paged_reserve(const PagedReserve& a, int num_sms, cudaStream_t stream) {
  const int smem = 2 * (a.B + 1) * static_cast<int>(sizeof(int));
  const long long work = static_cast<long long>(a.rows) / 4 + 1;
  const int grid = static_cast<int>(std::max<long long>(1, std::min<long long>(2 * num_sms, (work + kThreads - 1) / kThreads)));
  return launch_programmatic(reserve_kernel, dim3(grid), dim3(kThreads), smem, stream, a);
}

cudaError_t launch_paged_release(const PagedRelease& a, int num_sms, cudaStream_t stream) {
  const int smem = (a.B + 1) * static_cast<int>(sizeof(int));
  const long long work = static_cast<long long>(a.B) * a.max_pages;
  const int grid =
      static_cast<int>(std::max<long long>(1, std::min<long long>(num_sms, (work + 4 * kThreads - 1) / (4 * kThreads))));
  return launch_programmatic(release_kernel, dim3(grid), dim3(kThreads), smem, stream, a);
}

// ---------------------------------------------------------------------------
// Cache writes with rotary positions
// ---------------------------------------------------------------------------
// A CTA takes `tokens` tokens at a time. Its threads first load their share of
// the rows, then form the tokens' cosines and sines once for all heads (the
// angle in 64 bits, as turns, so its reduction is a subtraction; sincospif of
// the remainder), then turn and store. A thread's unit is 16 values of one
// head: two 16-byte chunks. With halves the unit holds both members of eight
// pairs (chunks c and c + pairs / 8), so it reads all it needs before it writes
// and q_out may be q itself.
template <bool ADJACENT>
__global__ void __launch_bounds__(kThreads) write_kernel(PagedWrite a) {
  grid_dep_launch();
  grid_dep_wait();
  __shared__ float2 turn[2][kWriteTurns];
  const int tid = threadIdx.x;
  const int lanes = a.d / 16;                    // units per head
  const int units = (a.Hq + 2 * a.Hkv) * lanes;  // per token (Hq = 0 without q)
  const int pc = a.pairs / 8;                    // chunks of the first members (halves)
  const float inv_units = 1.0f / static_cast<float>(units);
  constexpr int kPre = 4;
  const long long total_slots = static_cast<long long>(a.num_pages) << a.page_shift;
  int buf = 0;
  for (long long t0 = static_cast<long long>(blockIdx.x) * a.tokens; t0 < a.rows;
       t0 += static_cast<long long>(gridDim.x) * a.tokens, buf ^= 1) {
    const int nt = static_cast<int>(min(static_cast<long long>(a.tokens), a.rows - t0));
    const int all = nt * units;
    // Where unit u lives: its source row, its two chunks and its destination.
    struct Unit {
      const uint4* src;
      uint4* dst;
      int c0, c1, token;
      bool turned;
    };
    auto locate = [&](int u) {
      Unit r;
      r.token = static_cast<int>((static_cast<float>(u) + 0.5f) * inv_units);  // u / units (u < 2^16: exact)
      const int w = u - r.token * units;
      const int head = w / lanes, l = w - head * lanes;
      const long long t = t0 + r.token;
      const bool is_v = head >= a.Hq + a.Hkv;
      r.c0 = 2 * l;
      r.c1 = 2 * l + 1;
      r.turned = false;
      if (!is_v && a.pairs > 0) {
        if (ADJACENT) {
          r.turned = r.c0 * 4 < a.pairs;
        } else if (l < pc) {
          r.c0 = l;
          r.c1 = l + pc;
          r.turned = true;
        }
      }
      if (head < a.Hq) {
        r.src = reinterpret_cast<const uint4*>(a.q + t * a.q_stride + head * a.d);
        r.dst = reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + head * a.d);
      } else {
        const int h = is_v ? head - a.Hq - a.Hkv : head - a.Hq;
        r.src = reinterpret_cast<const uint4*>(is_v ? a.v + t * a.v_stride + h * a.d : a.k + t * a.k_stride + h * a.d);
        const int slot = a.slots[t];
        r.dst = nullptr;
        if (slot >= 0 && slot < total_slots) {
          const size_t row = ((static_cast<size_t>(slot >> a.page_shift) * a.Hkv + h) << a.page_shift) +
                             (slot & ((1 << a.page_shift) - 1));
          r.dst = reinterpret_cast<uint4*>((is_v ? a.v_cache : a.k_cache) + row * a.d);
        } else if (slot != -1) {
          raise_invalid(a.ws, 204);
        }
      }
      return r;
    };
    auto finish = [&](const Unit& r, uint4 x, uint4 y) {
      if (r.dst == nullptr) return;
      if (r.turned) {
        const float2* cs = turn[buf] + r.token * a.pairs;
        uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
        if (ADJACENT) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            xw[e] = turn_word(xw[e], cs[r.c0 * 4 + e]);
            yw[e] = turn_word(yw[e], cs[r.c1 * 4 + e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) turn_words(xw[e], yw[e], cs[r.c0 * 8 + 2 * e], cs[r.c0 * 8 + 2 * e + 1]);
        }
        x = make_uint4(xw[0], xw[1], xw[2], xw[3]);
        y = make_uint4(yw[0], yw[1], yw[2], yw[3]);
      }
      r.dst[r.c0] = x;
      r.dst[r.c1] = y;
    };
    Unit pre[kPre];
    uint4 px[kPre], py[kPre];
#pragma unroll
    for (int i = 0; i < kPre; ++i) {
      const int u = tid + i * kThreads;
      if (u < all) {
        pre[i] = locate(u);
        px[i] = pre[i].src[pre[i].c0];
        py[i] = pre[i].src[pre[i].c1];
      }
    }
    // Two buffers: a thread that is a round ahead writes the other one, and
    // the barrier below keeps it from getting two ahead.
    for (int i = tid; i < nt * a.pairs; i += kThreads) {
      const int tk = i / a.pairs, p = i - tk * a.pairs;
      int axis = a.pair_axis ? a.pair_axis[p] : 0;
      if (axis < 0 || axis >= a.axes) {
        raise_invalid(a.ws, 205);
        axis = 0;
      }
      const double pos = a.positions[static_cast<long long>(axis) * a.rows + t0 + tk];
      const double turns = pos * static_cast<double>(a.inv_freq[p]) * 0.15915494309189535;  // 1 / (2 pi)
      float sn, cn;
      sincospif(2.0f * static_cast<float>(turns - rint(turns)), &sn, &cn);
      turn[buf][i] = make_float2(cn, sn);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPre; ++i)
      if (tid + i * kThreads < all) finish(pre[i], px[i], py[i]);
    for (int u = tid + kPre * kThreads; u < all; u += kThreads) {
      const Unit r = locate(u);
      finish(r, r.src[r.c0], r.src[r.c1]);
    }
  }
}

cudaError_t launch_paged_write(PagedWrite a, int num_sms, cudaStream_t stream) {
  const int units = (a.Hq + 2 * a.Hkv) * (a.d / 16);
  a.tokens = std::max(1, std::min(kWriteTurns / std::max(a.d / 2, 1), 2 * kThreads / units));
  const int grid = static_cast<int>(
      std::max<long long>(1, std::min<long long>(8LL * num_sms, (static_cast<long long>(a.rows) + a.tokens - 1) / a.tokens)));
  return launch_programmatic(a.adjacent ? write_kernel<true> : write_kernel<false>, dim3(grid), dim3(kThreads), 0, stream, a);
}

}  // namespace sigattn
