// paged_many.cu -- sigmoid attention of many new tokens per sequence (prompts and
// chunks of prompts, beside any number of single tokens) over a paged cache.
//
//   o_i = sum_{j < N} sigma(q_i . k_j / sqrt(d) - ln N) v_j
//
// The arithmetic bounds it, so the products take the forward kernel's shape
// (fwd.cu): 128 query rows by 128 keys, S = Q K^T and O += P V with P read from
// tensor memory, two query tiles per CTA that share every K/V block, one
// issuing thread per tile. What differs:
//
//  * A tile's 128 rows are T = floor(128 / G) tokens times the G query heads
//    that share a key/value head, so shared heads read their keys once.
//  * Keys come from pages: the producer warp looks the page numbers up and its
//    lanes issue one box per page and 64 columns.
//  * Each row has its own N (causal): the bias is a register of the row's
//    thread, and only blocks past the tile's first row's N run masking code.
//    A tile stops at the last block that one of its rows sees.
//  * The work is shared out in equal runs of key blocks (paged_run.cuh): few
//    tiles over long texts are cut along the keys, and the causal triangle's
//    uneven tiles need no other balancing. Parts are fp32 sums, added in CTA
//    order by the CTA that stores last.
//
// Roles (19 warps): 0-15 epilogue (warps 0-7 tile 0, 8-15 tile 1; per tile, four
// warps for each half of a block's keys), 16 the producer, 17 and 18 the
// issuers of tiles 0 and 1.
// TMEM: S of tile t at columns [128t, 128t + 128), O at 256 + t D; P over S
// (d = 128) or in a region of its own after O (d = 64).
#include "paged_run.cuh"

namespace sigattn {

namespace {

template <int D>
struct ManyCfg {
  static constexpr int CH = D / 64;
  static constexpr int KST = (D == 128) ? 2 : 3;
  static constexpr int VST = (D == 128) ? 2 : 3;
  static constexpr int BOX_BYTES = 128 * 128;
  static constexpr int TILE_BYTES = CH * BOX_BYTES;
  static constexpr int OFF_K = 2 * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + KST * TILE_BYTES;
  static constexpr int SMEM_ALLOC = OFF_V + VST * TILE_BYTES + 1024;
  static constexpr bool SEP_P = (D == 64);
  static constexpr int TM_S = 0, TM_O = 256, TM_P = TM_O + 2 * D;
  static constexpr int TMEM_COLS = 512;
  static constexpr int EPI_WARPS = 16;
  static constexpr int THREADS = (EPI_WARPS + 3) * 32;
};

template <int KST, int VST>
struct ManyBarriers {
  uint64_t q_full, q_empty;
  uint64_t k_full[KST], k_empty[KST];
  uint64_t v_full[VST], v_empty[VST];
  uint64_t s_full[2], p_full[4], o_full[2], o_empty[2];
  uint64_t epi_done[2];  // tile t's warps finished their pass over a block (d = 128: the tiles take turns)
  uint64_t s_read[2];    // SEP_P: the epilogue copied tile t's S out of TMEM
  uint64_t pv_done[2];   // SEP_P: tile t's PV products of a block completed (P region free)
  uint64_t stored, counted, drain[2];
  SegRing ring;
  PlanRun run;
  uint32_t tmem_base;
  int abort, last;
};

// sum_{k < n} floor((x k + y) / 128), x and y >= 0: after taking out whole
// parts, the lattice points under the line are counted along the other axis.
__device__ __forceinline__ long long floor_sum(long long n, long long x, long long y) {
  long long m = kKeyBlock, sum = 0;
  while (n > 0) {
    if (x >= m) {
      sum += n * (n - 1) / 2 * (x / m);
      x %= m;
    }
    if (y >= m) {
      sum += n * (y / m);
      y %= m;
    }
    const long long top = x * n + y;
    if (top < m) break;
    n = top / m;
    y = top % m;
    const long long t = m;
    m = x;
    x = t;
  }
  return sum;
}

// Tiles of a sequence: an item is two query tiles, 2 T tokens.
struct TileMath {
  int item;  // tokens per item
  int causal;
  __device__ __forceinline__ int blocks(const SeqInfo& s, int k) const {
    return blocks(s.m, s.n, min((k + 1) * item, s.m) - 1);
  }
  __device__ __forceinline__ int items(const SeqInfo& s) const { return (s.m + item - 1) / item; }
  // Keys that token i sees.
  __device__ __forceinline__ int seen(int m, int n, int i) const {
    return causal ? max(0, min(n, n - m + i + 1)) : n;
  }
  // Blocks that tokens up to i of the chunk walk.
  __device__ __forceinline__ int blocks(int m, int n, int i) const { return seq_blocks(seen(m, n, i)); }
  // Blocks of items 0 .. k - 1 (k <= items).
  __device__ __forceinline__ long long before(const SeqInfo& s, int k) const {
    if (!causal) return static_cast<long long>(k) * seq_blocks(s.n);
    if (k == 0) return 0;
    long long sum = 0;
    if (k == items(s)) {  // the last item may hold fewer tokens
      sum = seq_blocks(s.n);
      --k;
    }
    // Item i's last token sees x(i) = n - m + (i + 1) item keys; where x <= 0
    // it walks the one block that writes its zeros.
    const long long c = static_cast<long long>(s.n) - s.m;
    const long long none = c < 0 ? min(static_cast<long long>(k), -c / item) : 0;
    return sum + none + floor_sum(k - none, item, c + (none + 1) * item + kKeyBlock - 1);
  }
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(ManyCfg<D>::THREADS, 1)
    paged_many_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PagedAttend a) {
  using C = ManyCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ ManyBarriers<C::KST, C::VST> bar;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bar.abort;
  int* ws = a.ws;
  constexpr int kProducer = C::EPI_WARPS, kIssuer = C::EPI_WARPS + 1;

  if (threadIdx.x == 0) {
    mbar_init(&bar.q_full, 1);
    mbar_init(&bar.q_empty, 2);
    for (int s = 0; s < C::KST; ++s) { mbar_init(&bar.k_full[s], 1); mbar_init(&bar.k_empty[s], 2); }
    for (int s = 0; s < C::VST; ++s) { mbar_init(&bar.v_full[s], 1); mbar_init(&bar.v_empty[s], 2); }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar.s_full[t], 1);
      mbar_init(&bar.p_full[2 * t], 4);
      mbar_init(&bar.p_full[2 * t + 1], 4);
      mbar_init(&bar.o_full[t], 1);
      mbar_init(&bar.o_empty[t], 8);
      mbar_init(&bar.epi_done[t], 8);
      mbar_init(&bar.s_read[t], 8);
      mbar_init(&bar.pv_done[t], 1);
      mbar_init(&bar.drain[t], 1);
    }
    mbar_init(&bar.stored, C::EPI_WARPS);
    mbar_init(&bar.counted, 1);
    seg_ring_init(bar.ring, C::EPI_WARPS + 2);
    bar.abort = 0;
    fence_mbar_init();
  }
  if (warp == kIssuer) {
    tmem_alloc(&bar.tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }
  const int G = a.Hq / a.Hkv;
  const int T = 128 / G;  // tokens per tile
  const TileMath math{2 * T, a.causal};
  grid_dep_launch();
  grid_dep_wait();
  plan_run<C::THREADS>(a, &bar.run, [&](const SeqInfo& s) { return math.before(s, math.items(s)); });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;

  // Tile t of a segment works on blocks [j0, end): none where it has no tokens
  // or its rows see none of them.
  auto tile_end = [&](const Segment& seg, int t) {
    const int i0 = seg.tile * 2 * T + t * T;
    if (i0 >= seg.m) return seg.j0;
    return max(seg.j0, min(seg.j1, math.blocks(seg.m, seg.n, min(i0 + T, seg.m) - 1)));
  };

  if (warp == kProducer) {
    // ------------------------------------------------------------- producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const int rb = min(1 << a.page_shift, kKeyBlock);  // keys per box
    uint32_t rst = 0, rph = 0, qph = 0;
    uint32_t st[2] = {0, 0}, ph[2] = {0, 0}, loads[2] = {0, 0};
    int q_last = -1;
    bool ok = true;
    RunWalker<TileMath> walk(a, math, bar.run, lane);
    const Segment& seg = walk.seg;
    for (bool more = bar.run.count > 0; ok && more; more = ok && walk.next()) {
      if (!(ok = seg_publish(bar.ring, rst, rph, seg, lane, abort_flag, ws, 400))) break;
      if (!(ok = warp_wait(&bar.q_empty, qph ^ 1, abort_flag, ws, 401))) break;
      if (lane == 0) {
        const int i0 = seg.tile * 2 * T, ntiles = i0 + T < seg.m ? 2 : 1;
        mbar_arrive_expect_tx(&bar.q_full, ntiles * T * G * 128 * C::CH);
        for (int t = 0; t < ntiles; ++t)
          for (int c = 0; c < C::CH; ++c)
            tma_load_3d(sQ + t * C::TILE_BYTES + c * C::BOX_BYTES, &tm_q, &bar.q_full, c * 64, seg.head * G,
                        seg.start + i0 + t * T);
      }
      q_last = static_cast<int>(qph);
      qph ^= 1;
      for (int j = seg.j0; ok && j < seg.j1; ++j) {
        const int keys = min(kKeyBlock, seg.n - j * kKeyBlock);
        const int boxes = (keys + rb - 1) / rb;  // 0 for a sequence without keys
        int row;
        const int z = walk.locate(j, lane / C::CH, rb, lane / C::CH < boxes, &row);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          uint64_t* full = kv ? &bar.v_full[st[1]] : &bar.k_full[st[0]];
          if (!(ok = warp_wait(kv ? &bar.v_empty[st[1]] : &bar.k_empty[st[0]], ph[kv] ^ 1, abort_flag, ws, 402))) break;
          if (lane == 0) mbar_arrive_expect_tx(full, boxes * rb * 128 * C::CH);
          __syncwarp();
          if (lane < boxes * C::CH)
            tma_load_3d((kv ? sV : sK) + st[kv] * C::TILE_BYTES + (lane % C::CH) * C::BOX_BYTES +
                            (lane / C::CH) * rb * 128,
                        kv ? &tm_v : &tm_k, full, (lane % C::CH) * 64, row, z);
          __syncwarp();
          ++loads[kv];
          if (++st[kv] == (kv ? C::VST : C::KST)) { st[kv] = 0; ph[kv] ^= 1; }
        }
      }
    }
    if (ok) ok = seg_publish(bar.ring, rst, rph, end_segment(), lane, abort_flag, ws, 403);
    if (!ok) {  // aborting: let the copies in flight land before the CTA exits
      int never = 0;
      volatile int* no_abort = &never;
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t slots = kv ? C::VST : C::KST;
        for (uint32_t x = 0; x < slots && x < loads[kv]; ++x) {
          const uint32_t idx = loads[kv] - 1 - x;
          mbar_wait(kv ? &bar.v_full[idx % slots] : &bar.k_full[idx % slots], (idx / slots) & 1, no_abort, nullptr, 0);
        }
      }
      if (q_last >= 0) mbar_wait(&bar.q_full, q_last, no_abort, nullptr, 0);
    }
  } else if (warp >= kIssuer) {
    // ------------------------------------------------------- issuer of tile t
    // Both issuers wait for every load and give an arrival on every "empty"
    // barrier, whether or not their tile works on the block. Lane 0 issues; the
    // whole warp walks along to zero the rows of V past a text's end.
    const int t = warp - kIssuer;
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
    const uint64_t d_q = smem_desc_sw128(smem_u32(sQ), 16, 1024) + ((t * C::TILE_BYTES) >> 4);
    const uint64_t d_k = smem_desc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t d_v = smem_desc_sw128(smem_u32(sV), C::BOX_BYTES, 1024);  // MN-major view of V
    constexpr uint64_t kTile = C::TILE_BYTES >> 4;
    const uint32_t tm_s = tmem + C::TM_S + t * 128;
    const uint32_t tm_o = tmem + C::TM_O + t * D;
    const uint32_t tm_p = C::SEP_P ? tmem + C::TM_P + t * 64 : tm_s;
    constexpr int kPHalf = C::SEP_P ? 32 : 64;
    uint32_t kst = 0, kph = 0, vst = 0, vph = 0, qph = 0, pph[2] = {0, 0}, oph = 0, srph = 0, rst = 0, rph = 0;
    bool s_pending = false;  // SEP_P: an S was issued whose copy-out has not been awaited
    bool ok = true;
    while (ok) {
      Segment seg;
      if (!(ok = seg_read<true>(bar.ring, rst, rph, &seg, abort_flag, ws, 410))) break;
      __syncwarp();
      seg_release(bar.ring, rst, rph, lane == 0);
      if (seg.j1 < 0) break;
      const int end = tile_end(seg, t);
      if (!(ok = warp_wait(&bar.q_full, qph, abort_flag, ws, 411))) break;
      qph ^= 1;
      auto take_k = [&](int j) -> bool {
        if (!warp_wait(&bar.k_full[kst], kph, abort_flag, ws, 412)) return false;
        if (j < end) {
          if (C::SEP_P && s_pending) {  // the epilogue must have copied the previous S out
            if (!warp_wait(&bar.s_read[t], srph, abort_flag, ws, 413)) return false;
            srph ^= 1;
          }
          s_pending = true;
          tc_fence_after();
          if (lane == 0) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = ((kk >> 2) * C::BOX_BYTES + (kk & 3) * 32) >> 4;
              mma_ss(tm_s, d_q + off, d_k + kst * kTile + off, idesc_s, kk > 0 ? 1u : 0u);
            }
            mma_commit(&bar.s_full[t]);
          }
        }
        if (lane == 0) {
          if (j + 1 == seg.j1) mma_commit(&bar.q_empty);
          mma_commit(&bar.k_empty[kst]);
        }
        __syncwarp();
        if (++kst == C::KST) { kst = 0; kph ^= 1; }
        return true;
      };
      auto take_v = [&](int j) -> bool {
        if (!warp_wait(&bar.v_full[vst], vph, abort_flag, ws, 414)) return false;
        if (j < end) {
          // The products take keys in sixteens: rows of V past the text's end in
          // the last sixteen are zeroed (their weights are 0, and 0 * NaN must
          // not be). Both issuers write the same zeros.
          const int keys = min(kKeyBlock, seg.n - j * kKeyBlock);
          const int steps = max(1, (keys + 15) / 16);
          if (keys < steps * 16) {
            uint4* v = reinterpret_cast<uint4*>(sV + vst * C::TILE_BYTES);
            for (int i = lane; i < (steps * 16 - keys) * 8; i += 32)
              for (int c = 0; c < C::CH; ++c) v[(c * C::BOX_BYTES + keys * 128) / 16 + i] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!warp_wait(&bar.p_full[2 * t + h], pph[h], abort_flag, ws, 415)) return false;
            pph[h] ^= 1;
            if (j == seg.j0 && h == 0) {
              if (!warp_wait(&bar.o_empty[t], oph ^ 1, abort_flag, ws, 416)) return false;
              oph ^= 1;
            }
            tc_fence_after();
            if (lane == 0) {
              const uint64_t b0 = d_v + vst * kTile + ((h * 64 * 128) >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (4 * h + kk < steps)
                  mma_ts(tm_o, tm_p + h * kPHalf + kk * 8, b0 + ((kk * 2048) >> 4), idesc_o,
                         (j > seg.j0 || h > 0 || kk > 0) ? 1u : 0u);
            }
          }
        }
        if (lane == 0) {
          mma_commit(&bar.v_empty[vst]);
          if (C::SEP_P && j < end) mma_commit(&bar.pv_done[t]);
        }
        __syncwarp();
        if (++vst == C::VST) { vst = 0; vph ^= 1; }
        return true;
      };
      if (!(ok = take_k(seg.j0))) break;
      for (int j = seg.j0; ok && j < seg.j1; ++j) {
        // S(j + 1) goes first where P has its own region; otherwise it
        // overwrites P(j) and follows PV(j).
        if (C::SEP_P && j + 1 < seg.j1 && !(ok = take_k(j + 1))) break;
        if (!(ok = take_v(j))) break;
        if (!C::SEP_P && j + 1 < seg.j1 && !(ok = take_k(j + 1))) break;
      }
      if (!ok) break;
      if (lane == 0 && seg.j0 < end) mma_commit(&bar.o_full[t]);
      __syncwarp();
    }
    if (lane == 0) {
      int never = 0;
      mma_commit(&bar.drain[t]);
      mbar_wait(&bar.drain[t], 0, &never, ws, 419);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- epilogue
    const int t = warp >> 3;                       // query tile of this warp
    const int h = (warp >> 2) & 1;                 // its half (64 keys) of each block
    const int r = ((warp & 3) << 5) + lane;        // row within the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) << 5) << 16;
    const uint32_t tS = tmem + lane_off + C::TM_S + t * 128 + h * 64;
    const uint32_t tP = C::SEP_P ? tmem + lane_off + C::TM_P + t * 64 + h * 32 : tS;
    const uint32_t tO = tmem + lane_off + C::TM_O + t * D + h * (D / 2);
    constexpr float scale_l2e = Scale<D>::value * kLog2e;
    const int ri = r / G, rg = r - ri * G;         // the row's token and head within the tile
    uint32_t sph = 0, oph = 0, turn_ph = 0, pvph = 0, rst = 0, rph = 0, parts = 0;
    bool pv_pending = false;  // SEP_P: a P was written whose PV has not been awaited
    bool turned = false;      // a block was shared with the other tile before
    bool ok = true;
    while (ok) {
      Segment seg;
      if (!(ok = seg_read<true>(bar.ring, rst, rph, &seg, abort_flag, ws, 420))) break;
      if (seg.j1 < 0) break;
      const int i0 = seg.tile * 2 * T + t * T;
      const int seg_j0 = seg.j0, end = tile_end(seg, t), other_end = tile_end(seg, 1 - t);
      const int i = i0 + ri;
      const bool row_ok = ri < T && i < seg.m;
      const int seen = math.seen(seg.m, seg.n, i);
      const float neg_log2n = -__log2f(static_cast<float>(max(seen, 1)));
      const int clear = math.seen(seg.m, seg.n, i0);  // keys that every row of the tile sees
      // Warps whose rows are all past the tile's last leave S and P alone
      // (what their rows of P hold reaches no other row).
      const bool idle = __all_sync(0xffffffffu, !row_ok);
      // One pass over key block j; the rows' masks only in MASKED passes.
      auto pass = [&](const int j, auto masked) -> bool {
        constexpr bool MASKED = decltype(masked)::value;
        if (!warp_wait(&bar.s_full[t], sph, abort_flag, ws, 421)) return false;
        sph ^= 1;
        // d = 128: the tiles take turns over the blocks that both work on (tile 1
        // follows tile 0 on each, tile 0 follows tile 1's previous one).
        const bool joint = !C::SEP_P && j < end && j < other_end;
        if (joint && (t == 1 || turned)) {
          if (!warp_wait(&bar.epi_done[1 - t], turn_ph, abort_flag, ws, 422)) return false;
          turn_ph ^= 1;
        }
        turned |= joint;
        tc_fence_after();
        if (!idle) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t s[32];
            tmem_ld32(tS + 32 * c, s);
            if (C::SEP_P && c == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar.s_read[t]);
            }
            uint32_t pk[16];
            if constexpr (MASKED) mask_scores(s, seen - (j * kKeyBlock + h * 64 + 32 * c), true);
            sigmoid32<false>(s, scale_l2e, neg_log2n, nullptr, row_ok);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              pk[e] = pack_bf16x2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
            // SEP_P: the P region is free once the tile's previous PV completed.
            if (C::SEP_P && c == 0 && pv_pending) {
              if (!warp_wait(&bar.pv_done[t], pvph, abort_flag, ws, 423)) return false;
              pvph ^= 1;
              tc_fence_after();
            }
            tmem_st16(tP + 16 * c, pk);
          }
          tmem_st_wait();
        } else if (C::SEP_P) {
          if (lane == 0) mbar_arrive(&bar.s_read[t]);
          if (pv_pending) {
            if (!warp_wait(&bar.pv_done[t], pvph, abort_flag, ws, 423)) return false;
            pvph ^= 1;
          }
        }
        pv_pending = true;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar.p_full[2 * t + h]);
          if (joint) mbar_arrive(&bar.epi_done[t]);  // hand the turn over
        }
        return true;
      };
      int j = seg_j0;
      const int plain = min(end, clear / kKeyBlock);  // blocks that every row sees whole
      for (; ok && j < plain; ++j) ok = pass(j, std::false_type{});
      for (; ok && j < end; ++j) ok = pass(j, std::true_type{});
      if (!ok) break;

      // The segment again, from the ring (its slot is released only below, so
      // that the passes need not keep it in registers).
      seg = seg_peek(bar.ring, rst);
      const bool whole = seg.j0 == 0 && seg.j1 == seg.blocks;
      const int token = seg.tile * 2 * T + t * T + ri;
      const bool writes = ri < T && token < seg.m;
      __nv_bfloat16* dst =
          a.o + (static_cast<size_t>(seg.start + token) * a.Hq + seg.head * G + rg) * D + h * (D / 2);
      constexpr size_t kPart = static_cast<size_t>(256) * D;
      const size_t mine = static_cast<size_t>(t * 128 + r) * D + h * (D / 2);
      // This warp's D / 2 columns of O, 32 at a time.
      if (seg.j0 < end) {
        if (!(ok = warp_wait(&bar.o_full[t], oph, abort_flag, ws, 424))) break;
        oph ^= 1;
        tc_fence_after();
        float* part = a.parts + (2 * blockIdx.x + (seg.j0 == 0)) * kPart + mine;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t v[32];
          tmem_ld32(tO + c * 32, v);
          if (c == D / 64 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.o_empty[t]);
          }
          if (!writes) continue;
          if (whole) store_row32(dst + c * 32, v, 1.0f);
          else store_row_f32(part + c * 32, v);
        }
      }
      if (!whole) {
        if (!(ok = last_part(&bar.stored, &bar.counted, &bar.last, seg, ws, warp, lane, parts, abort_flag, 425))) break;
        parts ^= 1;
      }
      if (!whole && bar.last) {
        // The sum of the tiles' parts. Lanes take four columns each, so a warp
        // reads SUB rows of a part at once, and it reads RB such rows (all of one
        // tile) before it adds any. The first part lies in its CTA's second
        // place, the others in their CTA's first; parts that start past the
        // tile's last block are not there.
        constexpr int LPR = D / 4, SUB = 32 / LPR, STEP = C::EPI_WARPS * SUB, RB = 128 / STEP;
        for (int u = 0; u < 2; ++u) {
          const int u0 = seg.tile * 2 * T + u * T;
          if (u0 >= seg.m) break;
          const int all = math.blocks(seg.m, seg.n, min(u0 + T, seg.m) - 1);
          const int row0 = warp * SUB + lane / LPR, used = min(T, seg.m - u0) * G;
          const float* from = a.parts + (2 * seg.first_cta + 1) * kPart + (u * 128 + row0) * D + 4 * (lane % LPR);
          float4 sum[RB];
#pragma unroll
          for (int k = 0; k < RB; ++k) sum[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int p = 0; p <= seg.last_cta - seg.first_cta; ++p) {
            if (p > 0 && p * bar.run.per - seg.lead >= all) break;
            float4 x[RB];
#pragma unroll
            for (int k = 0; k < RB; ++k) {
              x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (row0 + k * STEP < used) x[k] = __ldcg(reinterpret_cast<const float4*>(from + k * STEP * D));
            }
#pragma unroll
            for (int k = 0; k < RB; ++k) {
              sum[k].x += x[k].x;
              sum[k].y += x[k].y;
              sum[k].z += x[k].z;
              sum[k].w += x[k].w;
            }
            from += (p == 0 ? 1 : 2) * kPart;
          }
#pragma unroll
          for (int k = 0; k < RB; ++k) {
            const int row = row0 + k * STEP;
            if (row < used)
              *reinterpret_cast<uint2*>(
                  a.o + (static_cast<size_t>(seg.start + u0 + row / G) * a.Hq + seg.head * G + row % G) * D +
                  4 * (lane % LPR)) = make_uint2(pack_bf16x2(sum[k].x, sum[k].y), pack_bf16x2(sum[k].z, sum[k].w));
          }
        }
      }
      __syncwarp();
      seg_release(bar.ring, rst, rph, lane == 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

namespace {

template <int D>
cudaError_t launch_many_impl(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttend& a,
                             int grid, cudaStream_t stream) {
  using C = ManyCfg<D>;
  static PerDeviceOnce attr;
  const cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(paged_many_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
  });
  if (e != cudaSuccess) return e;
  return launch_programmatic(paged_many_kernel<D>, dim3(grid), dim3(C::THREADS), C::SMEM_ALLOC, stream, tq, tk, tv, a);
}

}  // namespace

cudaError_t launch_paged_many(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttend& a,
                              int grid, cudaStream_t stream) {
  return a.d == 64 ? launch_many_impl<64>(tq, tk, tv, a, grid, stream)
                   : launch_many_impl<128>(tq, tk, tv, a, grid, stream);
}

}  // namespace sigattn
