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
//    thread, and only blocks past the tile's first row's N are masked.
//    A tile stops at the last block that one of its rows sees.
//  * The work is shared out in equal runs of key blocks (paged_run.cuh): few
//    tiles over long texts are cut along the keys, and the causal triangle's
//    uneven tiles need no other balancing. Parts are fp32 sums, added in CTA
//    order by the CTA that stores last.
//  * Where a segment has one tile only (a single token beside other users'
//    prompts, a short chunk), its blocks alternate between the two tiles' S and
//    P regions and epilogue warps ("dual"): a lone tile would wait through the
//    chain S, weights, PV on every block. Issuer 0 then issues all products, so
//    that all of them add to one O in order.
//
// What bounds it: the chain of a tile's block, S, weights, PV. With two tiles in turn
// a block of both takes 4280 cycles, of which the weights' passes, one after the
// other, are 3500 (1024 each if the 16 MUFU lanes never waited); the tensor pipe is
// busy for 41 % of a call of two 4096-token prompts. On long calls the clock is held
// down by power besides. Two prompts of 4000 tokens behind 8192 to 16384 (16 heads of
// 128): 840 to 1025 us, 970 to 795 TFLOPS; 4096-token prompts, not causal: 543 us,
// 1010 TFLOPS. Short calls wait for their start (9000 cycles to the first load, half
// of them instruction misses) and for cut tiles' parts.
//
// Roles (20 warps): 0-15 epilogue (warps 0-7 tile 0, 8-15 tile 1; per tile, four
// warps for every other 32 of a block's keys), 16 and 17 the producers of K and
// of Q and V, 18 and 19 the issuers of tiles 0 and 1.
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
  static constexpr int QST = (D == 128) ? 3 : 4;  // query tiles: the next segment's are loaded ahead
  static constexpr int OFF_K = QST * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + KST * TILE_BYTES;
  static constexpr int SMEM_ALLOC = OFF_V + VST * TILE_BYTES + 1024;
  static constexpr bool SEP_P = (D == 64);
  static constexpr int TM_S = 0, TM_O = 256, TM_P = TM_O + 2 * D;
  static constexpr int TMEM_COLS = 512;
  static constexpr int EPI_WARPS = 16;
  static constexpr int THREADS = (EPI_WARPS + 4) * 32;
};

template <int QST, int KST, int VST, typename U>
struct ManyBarriers {
  uint64_t q_full[QST], q_empty[QST];
  uint64_t k_full[KST], k_empty[KST];
  uint64_t v_full[VST], v_empty[VST];
  uint64_t s_full[2], p_full[4], o_full[2], o_empty[2];
  uint64_t epi_done[2];  // tile t's warps finished their pass over a block (d = 128: the tiles take turns)
  uint64_t s_read[2];    // SEP_P: the epilogue copied tile t's S out of TMEM
  uint64_t pv_done[2];   // SEP_P: tile t's PV products of a block completed (P region free)
  uint64_t fin[2][4];    // issuer t's products of a segment completed (by segment, modulo 4)
  // Cut tiles of this CTA: [0] the run's first, if it began in another CTA's run and
  // ends in this one, [1] the run's last, if it goes on in the next CTA's.
  uint64_t stored[2], counted[2];
  uint64_t ask, answered;  // [1]: should its part be stored at all?
  uint64_t drain[2];
  Segment cut[2];
  int join[2];  // does this CTA add up the parts?
  int keep;     // [1]: the other parts were there, so this CTA's stayed in tensor memory
  SegRing ring;
  PlanRun<U> run;
  uint32_t tmem_base;
  int abort;
};

// The bf16 weights of 32 scores of one thread: sigma(x) for y = x log2(e) =
// s scale_l2e + neg_log2n. As in the whole-sequence kernels (sigmoid_n) a warp
// whose scores all lie in the far tail takes one exponential per weight. The
// general form here is 1 / (1 + 2^-y), one more MUFU operation where theirs is a
// polynomial: half the instructions, and instructions are what the short texts
// that come here wait for (eight sequences of 512 tokens: 82 -> 58 us); its relative
// error is that of an exponent in fp32 (1e-6 at 1000 keys, 4e-6 at 2^24) instead of
// 9e-4. The tail's three terms of the series leave out at most u^3 = 2.4e-4 of a weight
// at u = 1/16. Both are then rounded to bf16 (2^-8 of the weight at most): the second
// product's operands have one type, V's. Against 64 bits the output is off by 0.0023
// of its norm that way, of which its own rounding alone is 0.0017.
__device__ __forceinline__ void weights32(const uint32_t (&s)[32], float scale_l2e, float neg_log2n, bool lane_ok,
                                          uint32_t (&pk)[16]) {
  const uint64_t c1 = f2_splat(scale_l2e), c0 = f2_splat(neg_log2n - kTailY);
  uint64_t z[16];  // y - kTailY
  uint32_t all = 0xffffffffu;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    z[e] = f2_fma(f2_pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c1, c0);
    all &= static_cast<uint32_t>(z[e]) & static_cast<uint32_t>(z[e] >> 32);
  }
  if (__all_sync(0xffffffffu, (all >> 31) != 0 || !lane_ok)) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 zz = f2_unpack(z[e]);
      const uint64_t w = f2_pack(ex2_approx(zz.x), ex2_approx(zz.y));
      const uint64_t t = f2_fma(f2_fma(w, f2_splat(kTailC * kTailC * kTailC), f2_splat(-kTailC * kTailC)), w, f2_splat(kTailC));
      const float2 q = f2_unpack(f2_mul(t, w));
      pk[e] = pack_bf16x2(q.x, q.y);
    }
  } else {
    constexpr float k = 16.0f;  // 2^-kTailY
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 zz = f2_unpack(z[e]);
      const float2 d = f2_unpack(f2_fma(f2_pack(ex2_approx(-zz.x), ex2_approx(-zz.y)), f2_splat(k), f2_splat(1.0f)));
      pk[e] = pack_bf16x2(rcp_approx(d.x), rcp_approx(d.y));
    }
  }
}

// Where a segment's parts differ by its tiles. Two tiles: each works on the blocks
// that its rows see. One tile: "dual" from two blocks on, both sides take blocks
// in turn for the one tile; else side 0 works alone.
struct Shape {
  bool two, dual;
};

}  // namespace

// U: an unsigned type that holds the call's units of work.
template <int D, typename U>
__global__ void __launch_bounds__(ManyCfg<D>::THREADS, 1)
    paged_many_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PagedAttend a) {
  using C = ManyCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ ManyBarriers<C::QST, C::KST, C::VST, U> bar;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bar.abort;
  int* ws = a.ws;
  constexpr int kLoadK = C::EPI_WARPS, kLoadV = kLoadK + 1, kIssuer = kLoadK + 2;

  // The barriers, a few per warp: one thread would take 600 cycles over them.
  if (lane == 0 && warp < 7) {
    if (warp == 0) {
      for (int s = 0; s < C::QST; ++s) { mbar_init(&bar.q_full[s], 1); mbar_init(&bar.q_empty[s], 2); }
      bar.abort = 0;
    } else if (warp == 1) {
      for (int s = 0; s < C::KST; ++s) { mbar_init(&bar.k_full[s], 1); mbar_init(&bar.k_empty[s], 2); }
    } else if (warp == 2) {
      for (int s = 0; s < C::VST; ++s) { mbar_init(&bar.v_full[s], 1); mbar_init(&bar.v_empty[s], 2); }
    } else if (warp < 5) {
      const int t = warp - 3;
      mbar_init(&bar.s_full[t], 1);
      mbar_init(&bar.p_full[2 * t], 8);
      mbar_init(&bar.p_full[2 * t + 1], 8);
      mbar_init(&bar.o_full[t], 1);
      mbar_init(&bar.o_empty[t], 8);
      mbar_init(&bar.epi_done[t], 8);
      mbar_init(&bar.s_read[t], 8);
      mbar_init(&bar.pv_done[t], 1);
      mbar_init(&bar.drain[t], 1);
    } else if (warp == 5) {
      for (int s = 0; s < 4; ++s) { mbar_init(&bar.fin[0][s], 1); mbar_init(&bar.fin[1][s], 1); }
    } else {
      for (int k = 0; k < 2; ++k) { mbar_init(&bar.stored[k], C::EPI_WARPS); mbar_init(&bar.counted[k], 1); }
      mbar_init(&bar.ask, 1);
      mbar_init(&bar.answered, 1);
      seg_ring_init(bar.ring, C::EPI_WARPS + 2);
    }
    fence_mbar_init();
  }
  if (warp == kIssuer) {
    tmem_alloc(&bar.tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (lane == 0 && warp == kLoadK) tma_prefetch_desc(&tm_k);
  if (lane == 0 && warp == kLoadV) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_v);
  }
  const int G = a.Hq / a.Hkv;
  const int T = 128 / G;  // tokens per tile
  TileMath math{T, a.lone == 0, a.causal};
  grid_dep_launch();
  grid_dep_wait();
  auto units = [&](const SeqInfo& s) { return math.before<U>(s, math.items(s)); };
  auto joins = [&](const SeqInfo& s) {
    const float tiles = math.two(s, 0) ? 2.0f : 1.0f;
    return a.cut * 2.0f * tiles * static_cast<float>(min(s.m, math.item()) * G) * seq_blocks(s.n);
  };
  // Single tiles where that is at most a.lone units per CTA, else pairs.
  auto settled = [&](U total) { return math.pairs || total <= static_cast<U>(a.lone) * gridDim.x; };
  SeqWords words{};
  if (a.B <= kWarpPlan && (warp == kLoadK || warp == kLoadV)) words = seq_load(a, lane);
  if (a.B > kWarpPlan) {
    for (;; math.pairs = 1) {
      plan_run<C::THREADS>(a, 1 << math.pairs, &bar.run, units, joins);
      if (math.pairs) break;
      __syncthreads();
      if (settled(bar.run.total)) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;

  auto shape = [&](const Segment& seg) {
    const bool two = math.two(seg.m, seg.tile);
    return Shape{two, !two && seg.j1 - seg.j0 > 1};
  };
  // Does the CTA of a tile's first part look whether the rest is there before it
  // stores its own? (Not with more than two parts: all but the last come from
  // CTAs that do nothing else, and end together.)
  auto asks = [](const Segment& seg) { return seg.j0 == 0 && seg.last_cta == seg.first_cta + 1; };
  // Side t of a segment that is not dual works on blocks [j0, end): none where
  // its tile has no tokens or its rows see none of them.
  auto side_end = [&](const Segment& seg, int t) {
    const int i0 = seg.tile * math.item() + t * T;
    if (t == 1 && !math.two(seg.m, seg.tile)) return seg.j0;
    return max(seg.j0, min(seg.j1, math.blocks(seg.m, seg.n, min(i0 + T, seg.m) - 1)));
  };

  if (warp == kLoadK || warp == kLoadV) {
    // ------------------------------------- producers: segments and K; Q and V
    // Both walk the run; the K warp hands its segments to the other roles.
    const bool is_k = warp == kLoadK;
    PlanRun<U> run;
    if (a.B > kWarpPlan) {
      run = bar.run;
    } else {
      for (;; math.pairs = 1) {
        run = plan_warp<U>(a, words, 1 << math.pairs, units, joins);
        if (settled(run.total)) break;
      }
    }
    if (is_k && lane == 0) {  // (read by the other roles once they have a segment)
      bar.run.per = run.per;
      bar.run.pairs = math.pairs;
    }
    RunWalker<U, TileMath> walk(a, math, run, lane);
    const Segment& seg = walk.seg;
    TileRing<D> ring{is_k ? &tm_k : &tm_v, is_k ? sK : sV, is_k ? bar.k_full : bar.v_full, is_k ? bar.k_empty : bar.v_empty,
                     is_k ? C::KST : C::VST, 1 << walk.box_shift(), 0, 0, 0};
    uint32_t rst = 0, rph = 0, qst = 0, qph = 0, q_loads = 0;
    // Parts that this CTA has still to count (K warp; bits as in bar.cut). It counts
    // the first tile's between two loads, once they are stored, so that they cost the
    // epilogue its stores and no more (an epilogue that counts waits until the
    // stores of all SMs have drained, 9000 cycles). The last tile's it handles after
    // its last load: while the last products still run it looks whether the
    // other parts are there already. They mostly are, and then the epilogue
    // adds them to its own sum as it reads that from tensor memory, instead of
    // storing and reading it (both: two sequences of 4096 tokens of 16 heads 173 -> 167
    // us, eight of 512 tokens of 32 heads 56.8 -> 52.7 us).
    int cut = 0;
    auto count_part = [&](const int k) {
      if (lane == 0) {
        bar.join[k] = part_count(bar.cut[k], ws);
        mbar_arrive(&bar.counted[k]);
      }
      __syncwarp();
      cut &= ~(1 << k);
    };
    bool ok = true;
    while (ok && walk.advance()) {
      if (is_k) {
        const bool tail = seg.j1 < seg.blocks;
        if (lane == 0 && (tail || seg.j0 > 0)) bar.cut[tail ? 1 : 0] = seg;
        cut |= tail ? 2 : seg.j0 > 0 ? 1 : 0;
        if (!(ok = seg_publish(bar.ring, rst, rph, seg, lane, abort_flag, ws, 400))) break;
      } else {  // (here, since V is needed last)
        const int i0 = seg.tile * math.item(), ntiles = math.two(seg.m, seg.tile) ? 2 : 1;
        for (int t = 0; ok && t < ntiles; ++t) {
          if (!(ok = warp_wait(&bar.q_empty[qst], qph ^ 1, abort_flag, ws, 401))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bar.q_full[qst], T * G * 128 * C::CH);
            for (int c = 0; c < C::CH; ++c)
              tma_load_3d(sQ + qst * C::TILE_BYTES + c * C::BOX_BYTES, &tm_q, &bar.q_full[qst], c * 64, seg.head * G,
                          seg.start + i0 + t * T);
          }
          __syncwarp();
          ++q_loads;
          if (++qst == C::QST) { qst = 0; qph ^= 1; }
        }
      }
      for (int j = seg.j0; ok && j < seg.j1; ++j) {
        ok = ring.load(walk, j, lane, abort_flag, ws, is_k ? 402 : 404);
        if (j == seg.j0) walk.prefetch();
        if ((cut & 1) && __all_sync(0xffffffffu, mbar_test_wait(&bar.stored[0], 0))) count_part(0);
      }
    }
    if (ok && is_k) ok = seg_publish(bar.ring, rst, rph, end_segment(), lane, abort_flag, ws, 403);
    if (ok && (cut & 1) && (ok = warp_wait(&bar.stored[0], 0, abort_flag, ws, 426))) count_part(0);
    if (ok && (cut & 2)) {
      if (asks(bar.cut[1]) && (ok = warp_wait(&bar.ask, 0, abort_flag, ws, 427))) {
        if (lane == 0) {
          bar.keep = PartCount(bar.cut[1], ws).others();
          mbar_arrive(&bar.answered);
        }
        __syncwarp();
        if (bar.keep) cut = 0;
      }
      if (ok && cut != 0 && (ok = warp_wait(&bar.stored[1], 0, abort_flag, ws, 428))) count_part(1);
    }
    if (!ok) {
      ring.settle();
      int never = 0;
      for (uint32_t x = 0; x < C::QST && x < q_loads; ++x) {
        const uint32_t idx = q_loads - 1 - x;
        mbar_wait(&bar.q_full[idx % C::QST], (idx / C::QST) & 1, &never, nullptr, 0);
      }
    }
  } else if (warp >= kIssuer) {
    // ------------------------------------------------------- issuer of side t
    // Both issuers wait for every load and give an arrival on every "empty"
    // barrier (each sees every phase), whether or not their side works on the
    // block. One thread each: a tile's chain of S, weights and PV sets the pace,
    // and every warp-wide step in it costs (4450 cycles a block against 4200).
    const int t = warp - kIssuer;
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
      const uint64_t d_q = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t d_k = smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t d_v = smem_desc_sw128(smem_u32(sV), C::BOX_BYTES, 1024);  // MN-major view of V
      constexpr uint64_t kTile = C::TILE_BYTES >> 4;
      const uint32_t tm_o = tmem + C::TM_O + t * D;
      // Column of the weights of the kk-th sixteen keys of a block's half h. Where P
      // lies over S, each 32 keys' weights start where their scores did.
      auto p_at = [](const int h, const int kk) -> uint32_t {
        return C::SEP_P ? h * 32 + kk * 8 : h * 64 + (kk >> 1) * 32 + (kk & 1) * 8;
      };
      uint32_t kst = 0, kph = 0, vst = 0, vph = 0, qst = 0, qph = 0, oph = 0, rst = 0, rph = 0, segs = 0;
      // Per side e (bit e): parity of the blocks so far, and whether there were any.
      // Both issuers keep both sides' bits, since dual segments swap the issuer.
      uint32_t odd = 0, any = 0;
      bool was_two = false;  // the previous segment had two tiles
      bool ok = true;
      while (ok) {
        Segment seg;
        if (!(ok = seg_read<false>(bar.ring, rst, rph, &seg, abort_flag, ws, 410))) break;
        seg_release(bar.ring, rst, rph, true);
        if (seg.j1 < 0) break;
        math.pairs = bar.run.pairs;
        const Shape sh = shape(seg);
        const int end = side_end(seg, t);
        const int len = seg.j1 - seg.j0;
        // Side 1's regions change issuers between a segment of two tiles and a dual
        // one: the other issuer's products must have completed. (No issuer gets
        // four segments ahead of the other: the K ring is shorter.)
        if (segs > 0 && (t == 0 ? was_two && !sh.two : sh.two && !was_two) &&
            !(ok = role_wait(&bar.fin[1 - t][(segs - 1) & 3], ((segs - 1) >> 2) & 1, abort_flag, ws, 417)))
          break;
        uint64_t q_tile = 0;  // this side's query tile (dual: the only one)
        uint64_t* q_free = nullptr;
        for (int x = 0; x <= (sh.two ? 1 : 0); ++x) {
          if (!(ok = role_wait(&bar.q_full[qst], qph, abort_flag, ws, 411))) break;
          if (x == t) {
            q_tile = d_q + qst * kTile;
            q_free = &bar.q_empty[qst];
          } else {
            mbar_arrive(&bar.q_empty[qst]);
          }
          if (++qst == C::QST) { qst = 0; qph ^= 1; }
        }
        if (!ok) break;
        uint32_t fresh = 0;  // 1 once the segment's O holds a product
        // Block j's K and V. ALT: a dual segment, whose blocks alternate between the
        // sides; otherwise the side is this issuer's own and its addresses stay
        // put. `works`: whether it works on the block at all.
        auto take_k = [&](const int j, auto alt, const bool works) -> bool {
          if (!role_wait(&bar.k_full[kst], kph, abort_flag, ws, 412)) return false;
          if (works) {
            const int e = decltype(alt)::value ? (j - seg.j0) & 1 : t;
            // SEP_P: the epilogue must have copied the side's previous S out.
            if (C::SEP_P && (any >> e & 1) && !role_wait(&bar.s_read[e], (odd >> e & 1) ^ 1, abort_flag, ws, 413)) return false;
            odd ^= 1u << e;
            any |= 1u << e;
            tc_fence_after();
            const uint32_t tm_s = tmem + C::TM_S + e * 128;
            const uint64_t b0 = d_k + kst * kTile;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = ((kk >> 2) * C::BOX_BYTES + (kk & 3) * 32) >> 4;
              mma_ss(tm_s, q_tile + off, b0 + off, idesc_s, kk > 0 ? 1u : 0u);
            }
            mma_commit(&bar.s_full[e]);
          }
          if (j + 1 == seg.j1 && q_free != nullptr) mma_commit(q_free);
          mma_commit(&bar.k_empty[kst]);
          if (++kst == C::KST) { kst = 0; kph ^= 1; }
          return true;
        };
        uint32_t podd = odd;  // parity of the side's blocks before the one whose P is taken next
        auto take_v = [&](const int j, auto alt, const bool works) -> bool {
          if (!role_wait(&bar.v_full[vst], vph, abort_flag, ws, 414)) return false;
          const int e = decltype(alt)::value ? (j - seg.j0) & 1 : t;
          if (works) {
            // The products take keys in sixteens: rows of V past the text's end in
            // the last sixteen are zeroed (their weights are 0, and 0 * NaN must
            // not be). Both issuers write the same zeros.
            const int keys = min(kKeyBlock, seg.n - j * kKeyBlock);
            const int steps = max(1, (keys + 15) / 16);
            if (keys < steps * 16) {
              uint4* v = reinterpret_cast<uint4*>(sV + vst * C::TILE_BYTES);
              for (int i = 0; i < (steps * 16 - keys) * 8; ++i)
                for (int c = 0; c < C::CH; ++c) v[(c * C::BOX_BYTES + keys * 128) / 16 + i] = make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
            }
            const uint32_t tm_p = tmem + (C::SEP_P ? C::TM_P + e * 64 : C::TM_S + e * 128);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (!role_wait(&bar.p_full[2 * e + h], podd >> e & 1, abort_flag, ws, 415)) return false;
              if (fresh == 0 && h == 0) {
                if (!role_wait(&bar.o_empty[t], oph ^ 1, abort_flag, ws, 416)) return false;
                oph ^= 1;
              }
              tc_fence_after();
              const uint64_t b0 = d_v + vst * kTile + ((h * 64 * 128) >> 4);
              if (steps == 8) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_ts(tm_o, tm_p + p_at(h, kk), b0 + ((kk * 2048) >> 4), idesc_o, (h > 0 || kk > 0) ? 1u : fresh);
              } else {
                for (int kk = 0; kk < min(4, steps - 4 * h); ++kk)
                  mma_ts(tm_o, tm_p + p_at(h, kk), b0 + ((kk * 2048) >> 4), idesc_o, (h > 0 || kk > 0) ? 1u : fresh);
              }
            }
            podd ^= 1u << e;
            fresh = 1;
          }
          mma_commit(&bar.v_empty[vst]);
          if (C::SEP_P && works) mma_commit(&bar.pv_done[e]);
          if (++vst == C::VST) { vst = 0; vph ^= 1; }
          return true;
        };
        // S(j + 1) goes before PV(j) where its region is free of P(j): P has a region
        // of its own (d = 64), or the next block is the other side's (dual).
        // Otherwise S(j + 1) overwrites P(j) and follows PV(j).
        if (sh.dual) {
          const std::true_type alt{};
          const bool works = t == 0;
          ok = take_k(seg.j0, alt, works);
          for (int j = seg.j0; ok && j < seg.j1; ++j) {
            if (j + 1 < seg.j1) ok = take_k(j + 1, alt, works);
            ok = ok && take_v(j, alt, works);
          }
        } else {
          const std::false_type own{};
          ok = take_k(seg.j0, own, seg.j0 < end);
          for (int j = seg.j0; ok && j < seg.j1; ++j) {
            const bool works = j < end, next = j + 1 < seg.j1;
            if (C::SEP_P && next) ok = take_k(j + 1, own, j + 1 < end);
            ok = ok && take_v(j, own, works);
            if (!C::SEP_P && next) ok = ok && take_k(j + 1, own, j + 1 < end);
          }
        }
        if (!ok) break;
        if (fresh) mma_commit(&bar.o_full[t]);
        mma_commit(&bar.fin[t][segs & 3]);
        // The other side's blocks, or (dual, t = 1) both sides'.
        const int theirs = sh.dual ? (t == 1 ? len / 2 : 0) : side_end(seg, 1 - t) - seg.j0;
        odd ^= static_cast<uint32_t>(theirs & 1) << (sh.dual ? 1 : 1 - t);
        if (theirs > 0) any |= 1u << (sh.dual ? 1 : 1 - t);
        if (sh.dual && t == 1) {
          odd ^= static_cast<uint32_t>((len + 1) / 2 & 1);
          any |= 1u;
        }
        was_two = sh.two;
        ++segs;
      }
      int never = 0;
      mma_commit(&bar.drain[t]);
      mbar_wait(&bar.drain[t], 0, &never, ws, 419);
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int t = warp >> 3;                       // side of this warp
    const int h = (warp >> 2) & 1;                 // its 32 keys of each half of a block
    const int r = threadIdx.x & 127;               // row within the tile = TMEM lane
    const uint32_t quad = tmem + (static_cast<uint32_t>(r & 96) << 16);
    const uint32_t tS = quad + C::TM_S + t * 128 + h * 32;
    constexpr float scale_l2e = Scale<D>::value * kLog2e;
    uint32_t rst = 0, rph = 0;
    // Bits in one register (the passes leave few): parities of the waits for S, O,
    // the turn and PV; kPending: a P was written whose PV has not been
    // awaited (SEP_P); kTurned: a block was shared with the other tile before; kCut and
    // 2 kCut: a part of the run's first and last tile was stored; kKept: the last
    // tile's other parts are there.
    enum : uint32_t { kS = 1, kO = 2, kTurn = 4, kPv = 8, kPending = 16, kTurned = 32, kCut = 64, kKept = 256 };
    uint32_t bits = 0;
    // A part holds [tile][4 columns][row]: the lanes of a warp, which own rows,
    // write and read 512 bytes in a row.
    constexpr size_t kPart = static_cast<size_t>(256) * D;
    const size_t mine = static_cast<size_t>(t * 128) * D + (h * (D / 8) * 128 + r) * 4;
    auto row_of = [&](const Segment& s, const int token, const int of) {
      return a.o + (static_cast<size_t>(s.start + token) * a.Hq + s.head * G + r - of * G) * D + h * (D / 2);
    };
    bool ok = true;
    while (ok) {
      Segment seg;
      if (!(ok = seg_read<true>(bar.ring, rst, rph, &seg, abort_flag, ws, 420))) break;
      if (seg.j1 < 0) break;
      math.pairs = bar.run.pairs;
      const Shape sh = shape(seg);
      const int i0 = seg.tile * math.item() + (sh.dual ? 0 : t * T);
      // This side's blocks: from `j` on, every `step`-th, below `end`. Blocks below
      // `joint_end` are shared with the other tile.
      const int step = sh.dual ? 2 : 1;
      const int end = sh.dual ? seg.j1 : side_end(seg, t);
      int j = sh.dual ? seg.j0 + t : seg.j0;
      const int joint_end = (!C::SEP_P && sh.two) ? min(end, side_end(seg, 1 - t)) : 0;
      const int ri = r / G;  // the row's token within the tile
      const bool row_ok = ri < T && i0 + ri < seg.m;
      const int seen = math.seen(seg.m, seg.n, i0 + ri);
      const float neg_log2n = -__log2f(static_cast<float>(max(seen, 1)));
      const int clear = math.seen(seg.m, seg.n, i0);  // keys that every row of the tile sees
      // Warps whose rows are all past the tile's last leave S and P alone
      // (what their rows of P hold reaches no other row).
      const bool idle = __all_sync(0xffffffffu, !row_ok);
      const int plain = min(end, clear / kKeyBlock);  // blocks that every row sees whole
      // One pass over key block j: a chunk of 32 keys from each half of the block,
      // so that the product with the first half's weights runs while the second
      // half's are computed (8 prompts of 512 tokens 57.6 -> 56.7 us, 24 short chunks
      // at d = 64 18.1 -> 16.9 us against a half of the keys per warp; computing S in
      // halves as well, so that the next block's first starts after that product,
      // loses: 59.4 us). How often this code exists decides how short
      // texts run, whose passes wait for instructions (the forward kernel's
      // instances for masked and unmasked blocks with both chunks unrolled: 4500
      // cycles for a chunk instead of 800). At d = 128 one copy serves both chunks
      // and masked blocks too (kEither); at d = 64, where the passes set the pace,
      // masked blocks have a copy of their own and the chunks are unrolled
      // (4096-token prompts: 133 us, with one copy 154 us).
      enum : int { kPlain, kMasked, kEither };
      auto pass = [&](const int j, auto mode) -> bool {
        constexpr int MODE = decltype(mode)::value;
        if (!warp_wait(&bar.s_full[t], (bits & kS) != 0, abort_flag, ws, 421)) return false;
        bits ^= kS;
        // d = 128: the tiles take turns over the blocks that both work on (tile 1
        // follows tile 0 on each, tile 0 follows tile 1's previous one).
        const bool joint = !C::SEP_P && j < joint_end;
        if (joint) {
          if (t == 1 || (bits & kTurned)) {
            if (!warp_wait(&bar.epi_done[1 - t], (bits & kTurn) != 0, abort_flag, ws, 422)) return false;
            bits ^= kTurn;
          }
          bits |= kTurned;
        }
        tc_fence_after();
        if (!idle) {
#pragma unroll (C::SEP_P ? 2 : 1)
          for (int c = 0; c < 2; ++c) {
            uint32_t s[32];
            tmem_ld32(tS + 64 * c, s);
            if (C::SEP_P && c == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar.s_read[t]);
            }
            if (MODE == kMasked || (MODE == kEither && j >= plain)) {
              // One bit per key: tests of a word's bits go to predicates several at a
              // time, where 32 comparisons with `seen` take one instruction each.
              const int left = seen - (j * kKeyBlock + 64 * c + 32 * h);
              const uint32_t keep = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(keep & (1u << e))) s[e] = 0xff800000u;  // -inf: weight 0
            }
            uint32_t pk[16];
            weights32(s, scale_l2e, neg_log2n, row_ok, pk);
            // SEP_P: the P region is free once the tile's previous PV completed.
            if (C::SEP_P && c == 0 && (bits & kPending)) {
              if (!warp_wait(&bar.pv_done[t], (bits & kPv) != 0, abort_flag, ws, 423)) return false;
              bits ^= kPv;
              tc_fence_after();
            }
            tmem_st16(C::SEP_P ? quad + C::TM_P + t * 64 + c * 32 + h * 16 : tS + 64 * c, pk);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_full[2 * t + c]);
          }
        } else if (C::SEP_P) {
          if (lane == 0) mbar_arrive(&bar.s_read[t]);
          if (bits & kPending) {
            if (!warp_wait(&bar.pv_done[t], (bits & kPv) != 0, abort_flag, ws, 423)) return false;
            bits ^= kPv;
          }
        }
        if (C::SEP_P) bits |= kPending;
        if (lane == 0) {
          if (idle) {
            mbar_arrive(&bar.p_full[2 * t]);
            mbar_arrive(&bar.p_full[2 * t + 1]);
          }
          if (joint) mbar_arrive(&bar.epi_done[t]);  // hand the turn over
        }
        return true;
      };
      if constexpr (C::SEP_P) {
        for (; ok && j < plain; j += step) ok = pass(j, std::integral_constant<int, kPlain>{});
        for (; ok && j < end; j += step) ok = pass(j, std::integral_constant<int, kMasked>{});
      } else {
        for (; ok && j < end; j += step) ok = pass(j, std::integral_constant<int, kEither>{});
      }
      if (!ok) break;

      // The segment again, from the ring (its slot is released only below, so
      // that the passes need not keep it in registers).
      seg = seg_peek(bar.ring, rst);
      const Shape out = shape(seg);
      const bool holds = out.dual ? t == 0 : seg.j0 < side_end(seg, t);  // this side's O holds a sum
      const bool whole = seg.j0 == 0 && seg.j1 == seg.blocks, tail = seg.j1 < seg.blocks;
      if (tail && asks(seg)) {
        if (warp == 0 && lane == 0) mbar_arrive(&bar.ask);
        if (!(ok = warp_wait(&bar.answered, 0, abort_flag, ws, 429))) break;
        if (bar.keep) bits |= kKept;
      }
      const int of = r / G, token = seg.tile * math.item() + t * T + of;
      const bool writes = (t == 0 || out.two) && of < T && token < seg.m;
      // This warp's D / 2 columns of O, 32 at a time.
      if (holds) {
        if (!(ok = warp_wait(&bar.o_full[t], (bits & kO) != 0, abort_flag, ws, 424))) break;
        bits ^= kO;
        tc_fence_after();
      }
      if (holds && !(bits & kKept)) {
        __nv_bfloat16* dst = row_of(seg, token, of);
        float* part = a.parts + (2 * blockIdx.x + (seg.j0 == 0)) * kPart + mine;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t v[32];
          tmem_ld32(quad + C::TM_O + t * D + h * (D / 2) + c * 32, v);
          if (c == D / 64 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.o_empty[t]);
          }
          if (!writes) continue;
          if (whole) {
            store_row32(dst + c * 32, v, 1.0f);
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              __stcg(reinterpret_cast<uint4*>(part + (c * 8 + q) * 512),
                     make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
          }
        }
      }
      __syncwarp();
      if (!whole && !(bits & kKept)) {
        bits |= tail ? 2 * kCut : kCut;
        if (lane == 0) mbar_arrive(&bar.stored[tail ? 1 : 0]);
      }
      seg_release(bar.ring, rst, rph, lane == 0);
    }

    // The cut tiles that this CTA adds up: those whose parts it completed.
    for (int k = 0; ok && k < 2; ++k) {
      const bool kept = k == 1 && (bits & kKept);
      if (!kept) {
        if (!(bits & (kCut << k))) continue;
        if (!(ok = warp_wait(&bar.counted[k], 0, abort_flag, ws, 425))) break;
        if (!bar.join[k]) continue;
      }
      const Segment seg = bar.cut[k];
      const Shape sh = shape(seg);
      const int of = r / G, token = seg.tile * math.item() + t * T + of;
      const bool writes = (t == 0 || sh.two) && of < T && token < seg.m;
      __nv_bfloat16* dst = row_of(seg, token, of);
      // The first part lies in its CTA's second place, or if it was kept in tensor
      // memory, the others in their CTA's first. Parts that start past the
      // tile's last block are not there.
      const int i0 = seg.tile * math.item() + t * T;
      const int all = writes ? math.blocks(seg.m, seg.n, min(i0 + T, seg.m) - 1) : 0;
      int np = 1;
      while (np <= seg.last_cta - seg.first_cta && part_begin(seg, np, bar.run.per, sh.two ? 1 : 0) < all) ++np;
      const float* from = a.parts + (2 * seg.first_cta + 1) * kPart + mine;
      for (int c = 0; c < D / 32; ++c, from += 4 * 512) {
        float4 sum[4];
        if (kept) {
          uint32_t v[16];
          __syncwarp();
          tmem_ld16(quad + C::TM_O + t * D + h * (D / 2) + c * 16, v);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            sum[q] = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                                 __uint_as_float(v[4 * q + 3]));
        } else if (writes) {
#pragma unroll
          for (int q = 0; q < 4; ++q) sum[q] = __ldcg(reinterpret_cast<const float4*>(from + q * 512));
        }
        if (!writes) continue;
#pragma unroll 2
        for (int p = 1; p < np; ++p) {
          float4 x[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            x[q] = __ldcg(reinterpret_cast<const float4*>(from + (2 * p - 1) * kPart + q * 512));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            sum[q].x += x[q].x;
            sum[q].y += x[q].y;
            sum[q].z += x[q].z;
            sum[q].w += x[q].w;
          }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
          *reinterpret_cast<uint4*>(dst + c * 16 + q * 8) =
              make_uint4(pack_bf16x2(sum[2 * q].x, sum[2 * q].y), pack_bf16x2(sum[2 * q].z, sum[2 * q].w),
                         pack_bf16x2(sum[2 * q + 1].x, sum[2 * q + 1].y),
                         pack_bf16x2(sum[2 * q + 1].z, sum[2 * q + 1].w));
      }
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

template <int D, typename U>
cudaError_t launch_many_impl(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttend& a,
                             int grid, cudaStream_t stream) {
  using C = ManyCfg<D>;
  static PerDeviceOnce attr;
  const cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(paged_many_kernel<D, U>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
  });
  if (e != cudaSuccess) return e;
  return launch_programmatic(paged_many_kernel<D, U>, dim3(grid), dim3(C::THREADS), C::SMEM_ALLOC, stream, tq, tk, tv, a);
}

}  // namespace

cudaError_t launch_paged_many(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttend& a,
                              bool wide, int grid, cudaStream_t stream) {
  using W = unsigned long long;
  if (a.d == 64)
    return wide ? launch_many_impl<64, W>(tq, tk, tv, a, grid, stream) : launch_many_impl<64, uint32_t>(tq, tk, tv, a, grid, stream);
  return wide ? launch_many_impl<128, W>(tq, tk, tv, a, grid, stream) : launch_many_impl<128, uint32_t>(tq, tk, tv, a, grid, stream);
}

}  // namespace sigattn
