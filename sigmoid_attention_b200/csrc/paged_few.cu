// paged_few.cu -- sigmoid attention of a few new tokens per sequence over a
// paged cache (at most 64 query rows per key/value head, 32 at d = 128: G query
// heads times the new tokens).
//
//   o_i = sum_{j < N} sigma(q_i . k_j / sqrt(d) - ln N) v_j
//
// So few rows leave the work bound by reading K and V once. What that needs:
// every SM reads all the time, whatever the lengths are, and the arithmetic
// on a block keeps out of the way of the reads.
//
//  * Split. The unit of work is a block of 128 keys of one (sequence, key/value
//    head). All units of the call stand in one line (sequences, heads,
//    blocks), which is cut into equal runs, one per CTA: a run ends inside
//    a text where the cut falls, so ragged batches and single long texts
//    load the SMs alike. Weights of a sigmoid carry no row maximum or sum, so the
//    parts of a text cut over CTAs just add up: each stores fp32 partial
//    sums, and the CTA that stores last adds them in CTA order (fixed, so a
//    repeated call gives the same bits) and rounds once.
//  * The CTAs find their runs themselves, with one prefix sum over the batch's
//    lengths; there is no plan launch.
//  * Orientation. The keys are the 128 rows of the products, the queries the
//    columns: S^T = K Q^T (128 x NR) and O^T += V^T P^T (D x NR), NR = 16, 32 or
//    64. A product's time follows its columns, so a block costs an eighth to a
//    half of what it would with the queries padded to 128 rows, and each
//    epilogue thread owns one key: its NR weights go to shared memory as one
//    row of the second product's B operand.
//
//  * A thread issues a tcgen05.mma only about every 100 cycles, so a block's
//    eight O^T products cost 1400 cycles with their waits, which is what a
//    block of D = 64 takes to arrive. Blocks therefore alternate between two
//    groups, each with its own S^T region, P buffer, issuer and O^T
//    accumulator; a segment's two accumulators are added when it is read out.
//  * Reading a segment out (and joining a cut tile) is the work of four more
//    warps, so the next segment's weights do not wait for it: short texts
//    took 4200 cycles per segment before, most of them this chain.
//
// Bound by HBM: 64 texts of 256 to 8192 tokens, 32 query heads on 8, d = 128,
// 16-token pages: 116 us, 6.2 TB/s of 6.57 (a copy's rate); four texts of 100 to 262
// thousand tokens 189 us, 6.7 TB/s. Short calls are bound by latency: one token over
// 1000 keys 7.7 us, of which 2.6 lie before the first load (lengths, then pages,
// then the load, each a trip to memory) and 2 after the last product (parts
// stored, counted, added up).
//
// Roles (17 warps): 0-7 weights, four per group (thread = key), 8-11 output
// (thread = column of O), 12 and 13 the producers of K and of Q and V, 14 the
// issuer of S^T, 15 and 16 the groups' issuers of O^T.
#include "paged_run.cuh"

namespace sigattn {

namespace {

template <int D, int NR>
struct FewCfg {
  static constexpr int CH = D / 64;                     // 64-column chunks of a row
  static constexpr int BOX_BYTES = kKeyBlock * 128;    // [128 keys][64 columns]
  static constexpr int TILE_BYTES = CH * BOX_BYTES;
  // About 150 KB of K and V tiles are on the way or in use. K and V have rings
  // of their own: a slot is then awaited by one role only, which sees each
  // of its phases (a role that skipped one could take an earlier phase of the
  // same parity for the one it waits for). V tiles stay longer: they wait for P.
  static constexpr int KST = D == 64 ? 4 : 2;
  static constexpr int VST = D == 64 ? 5 : 3;
  static constexpr int STAGES = KST + VST;
  static constexpr int Q_CHUNK = NR * 128;
  static constexpr int Q_BYTES = CH * Q_CHUNK;
  static constexpr int QST = NR == 16 ? 4 : 2;          // segments' queries loaded ahead
  static constexpr int P_BYTES = kKeyBlock * 128;      // rows of 64 columns, NR of them in use
  static constexpr int OFF_P = STAGES * TILE_BYTES;
  static constexpr int OFF_Q = OFF_P + 2 * P_BYTES;
  static constexpr int OFF_RED = OFF_Q + QST * Q_BYTES;   // slices' sums of four rows of a join
  static constexpr int LPR = D / 4, SUB = 32 / LPR;     // lanes per row of a part, rows a warp reads at once
  static constexpr int OUT_WARPS = 4;
  static constexpr int SLICES = OUT_WARPS * SUB, RC = 4;
  static constexpr int RED_BYTES = SLICES * RC * LPR * 16;
  static constexpr int SMEM_ALLOC = OFF_RED + RED_BYTES + 1024;
  static_assert(SMEM_ALLOC <= 220 * 1024, "shared memory budget");
  static constexpr int TM_S = 0;                        // two S^T regions, then two O^T pairs
  static constexpr int TM_O = 2 * NR;
  static constexpr int TMEM_COLS = NR == 16 ? 128 : NR == 32 ? 256 : 512;  // >= 6 NR
  static constexpr int EPI_WARPS = 8;
  static constexpr int kLoadK = EPI_WARPS + OUT_WARPS, kLoadV = kLoadK + 1, kIssueS = kLoadK + 2, kIssueO = kLoadK + 3;
  static constexpr int THREADS = (kIssueO + 2) * 32;
};

template <int STAGES, int QST, typename U>
struct FewBarriers {
  uint64_t full[STAGES], empty[STAGES];  // K slots first, then V slots
  uint64_t q_full[QST], q_empty[QST];
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2], p_empty[2];
  uint64_t o_full[2], o_empty[2];
  uint64_t stored, counted, joined, drain[3];
  SegRing ring;
  PlanRun<U> run;
  uint32_t tmem_base;
  int abort, last;
};

}  // namespace

// U: an unsigned type that holds the call's units of work.
template <int D, int NR, typename U>
__global__ void __launch_bounds__(FewCfg<D, NR>::THREADS, 1)
    paged_few_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const PagedAttend a) {
  using C = FewCfg<D, NR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ FewBarriers<C::STAGES, C::QST, U> bar;
  __shared__ float s_log2n[C::EPI_WARPS][NR];  // each epilogue warp's log2 N and N of the segment's rows
  __shared__ int s_seen[C::EPI_WARPS][NR];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sP = smem + C::OFF_P;
  uint8_t* sQ = smem + C::OFF_Q;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &bar.abort;
  int* ws = a.ws;
  constexpr int kLoadK = C::kLoadK, kLoadV = C::kLoadV, kIssueS = C::kIssueS, kIssueO = C::kIssueO;

  // The barriers, a few per warp: one thread would take 500 cycles over them.
  if (lane == 0 && warp < 5) {
    if (warp == 0) {
      for (int s = 0; s < C::STAGES; ++s) mbar_init(&bar.full[s], 1);
      bar.abort = 0;
    } else if (warp == 1) {
      for (int s = 0; s < C::STAGES; ++s) mbar_init(&bar.empty[s], s < C::KST ? 1 : 2);
    } else if (warp < 4) {
      const int s = warp - 2;
      for (int i = s; i < C::QST; i += 2) { mbar_init(&bar.q_full[i], 1); mbar_init(&bar.q_empty[i], 1); }
      mbar_init(&bar.s_full[s], 1);
      mbar_init(&bar.s_empty[s], 4);
      mbar_init(&bar.p_full[s], 4);
      mbar_init(&bar.p_empty[s], 1);
      mbar_init(&bar.o_full[s], 2);
      mbar_init(&bar.o_empty[s], C::OUT_WARPS);
    } else {
      for (int s = 0; s < 3; ++s) mbar_init(&bar.drain[s], 1);
      mbar_init(&bar.stored, C::OUT_WARPS);
      mbar_init(&bar.counted, 1);
      mbar_init(&bar.joined, C::OUT_WARPS);
      seg_ring_init(bar.ring, C::EPI_WARPS + C::OUT_WARPS + 3);
    }
    fence_mbar_init();
  }
  if (warp == kIssueO) {
    tmem_alloc(&bar.tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (lane == 0 && warp == kLoadK) tma_prefetch_desc(&tm_k);
  if (lane == 0 && warp == kLoadV) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_v);
  }
  const int G = a.Hq / a.Hkv;
  grid_dep_launch();
  grid_dep_wait();
  auto units = [](const SeqInfo& s) -> U { return seq_blocks(s.n); };
  auto joins = [&](const SeqInfo& s) { return a.cut * static_cast<float>(s.m * G) * seq_blocks(s.n); };
  SeqWords words{};
  if (a.B <= kWarpPlan && (warp == kLoadK || warp == kLoadV)) words = seq_load(a, lane);
  if (a.B > kWarpPlan) plan_run<C::THREADS>(a, 1, &bar.run, units, joins);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem_base;

  if (warp == kLoadK || warp == kLoadV) {
    // ------------------------------------- producers: segments and K; Q and V
    // Both walk the run; the K warp hands its segments to the other roles.
    const bool is_k = warp == kLoadK;
    const OneTile tiles{};
    const PlanRun<U> run = a.B > kWarpPlan ? bar.run : plan_warp<U>(a, words, 1, units, joins);
    RunWalker<U, OneTile> walk(a, tiles, run, lane);
    const Segment& seg = walk.seg;
    TileRing<D> ring{is_k ? &tm_k : &tm_v, smem + (is_k ? 0 : C::KST * C::TILE_BYTES), bar.full + (is_k ? 0 : C::KST),
                     bar.empty + (is_k ? 0 : C::KST), is_k ? C::KST : C::VST, 1 << walk.box_shift(), 0, 0, 0};
    const int q_bytes = min(a.max_q * G, NR) * 128 * C::CH;
    uint32_t qb = 0, qph = 0, rst = 0, rph = 0, q_used = 0;
    bool ok = true;
    while (ok && walk.advance()) {
      if (is_k) {
        if (!(ok = seg_publish(bar.ring, rst, rph, seg, lane, abort_flag, ws, 300))) break;
      } else {  // (Q beside V, which is needed last, and several ahead, so that a wait for room
                // holds up no keys: draft tokens over 64 to 4096 keys 27.7 -> 24.9 us)
        if (!(ok = warp_wait(&bar.q_empty[qb], qph ^ 1, abort_flag, ws, 301))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar.q_full[qb], q_bytes);
          for (int c = 0; c < C::CH; ++c)
            tma_load_3d(sQ + qb * C::Q_BYTES + c * C::Q_CHUNK, &tm_q, &bar.q_full[qb], c * 64, seg.head * G, seg.start);
        }
        ++q_used;
        if (++qb == C::QST) { qb = 0; qph ^= 1; }
      }
      for (int j = seg.j0; ok && j < seg.j1; ++j) {
        ok = ring.load(walk, j, lane, abort_flag, ws, is_k ? 302 : 304);
        if (j == seg.j0) walk.prefetch();
      }
    }
    if (ok && is_k) ok = seg_publish(bar.ring, rst, rph, end_segment(), lane, abort_flag, ws, 303);
    if (!ok) {
      ring.settle();
      int never = 0;
      for (uint32_t s = 0; s < C::QST && s < q_used; ++s)
        mbar_wait(&bar.q_full[(q_used - 1 - s) % C::QST], ((q_used - 1 - s) / C::QST) & 1, &never, nullptr, 0);
    }
  } else if (warp == kIssueS) {
    // ------------------------------------------------- S^T = K Q^T (128 x NR)
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, NR, false, false);
      const uint64_t d_k = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t d_q = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      uint32_t st = 0, ph = 0, qb = 0, qph = 0, sb = 0, sph = 0, rst = 0, rph = 0;
      bool ok = true;
      while (ok) {
        Segment seg;
        if (!(ok = seg_read<false>(bar.ring, rst, rph, &seg, abort_flag, ws, 310))) break;
        seg_release(bar.ring, rst, rph, true);
        if (seg.j1 < 0) break;
        if (!(ok = role_wait(&bar.q_full[qb], qph, abort_flag, ws, 311))) break;
        for (int j = seg.j0; j < seg.j1; ++j) {
          if (!(ok = role_wait(&bar.full[st], ph, abort_flag, ws, 312))) break;
          if (!(ok = role_wait(&bar.s_empty[sb], sph ^ 1, abort_flag, ws, 313))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + C::TM_S + sb * NR, d_k + ((st * C::TILE_BYTES + (kk >> 2) * C::BOX_BYTES + (kk & 3) * 32) >> 4),
                   d_q + ((qb * C::Q_BYTES + (kk >> 2) * C::Q_CHUNK + (kk & 3) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
          mma_commit(&bar.s_full[sb]);
          mma_commit(&bar.empty[st]);
          if (j + 1 == seg.j1) mma_commit(&bar.q_empty[qb]);
          if ((sb ^= 1) == 0) sph ^= 1;
          if (++st == C::KST) { st = 0; ph ^= 1; }
        }
        if (++qb == C::QST) { qb = 0; qph ^= 1; }
      }
      int never = 0;
      mma_commit(&bar.drain[0]);
      mbar_wait(&bar.drain[0], 0, &never, ws, 319);
    }
  } else if (warp >= kIssueO) {
    // -------------------------------- O^T += V^T P^T (D x NR), group g's blocks
    // Both issuers wait for every V tile and release it (so each sees every
    // phase of a slot); the block's group uses it. At D = 64 the product's 128 rows
    // hold V's 64 columns twice (the second column block's distance is 0); the
    // second half is not read.
    const uint32_t g = warp - kIssueO;
    constexpr uint32_t idesc = idesc_bf16_f32(128, NR, true, true);
    const uint64_t d_v = smem_desc_sw128(smem_u32(smem), D == 64 ? 0 : C::BOX_BYTES, 1024);
    const uint64_t d_p = smem_desc_sw128(smem_u32(sP), C::P_BYTES, 1024) + ((g * C::P_BYTES) >> 4);
    uint32_t st = C::KST, ph = 0, t = 0, pph = 0, ob = 0, oph = 0, rst = 0, rph = 0;
    bool ok = true;
    while (ok) {
      Segment seg;
      if (!(ok = seg_read<true>(bar.ring, rst, rph, &seg, abort_flag, ws, 320))) break;
      __syncwarp();
      seg_release(bar.ring, rst, rph, lane == 0);
      if (seg.j1 < 0) break;
      if (!(ok = warp_wait(&bar.o_empty[ob], oph ^ 1, abort_flag, ws, 323))) break;
      const uint32_t tm_o = tmem + C::TM_O + (2 * ob + g) * NR;
      uint32_t fresh = 0;  // 1 once the segment's accumulator holds a product
      for (int j = seg.j0; j < seg.j1; ++j, ++t) {
        if (!(ok = warp_wait(&bar.full[st], ph, abort_flag, ws, 321))) break;
        if ((t & 1) == g) {
          // The product takes keys in sixteens. Rows of V past the text's end in
          // the last sixteen hold whatever the page (or an earlier tile) held;
          // their weights are 0, and 0 * NaN must not be: they are zeroed.
          const int keys = min(kKeyBlock, seg.n - j * kKeyBlock);
          const int steps = max(1, (keys + 15) / 16);
          if (keys < steps * 16) {
            uint4* v = reinterpret_cast<uint4*>(smem + st * C::TILE_BYTES);
            for (int i = lane; i < (steps * 16 - keys) * 8; i += 32)
              for (int c = 0; c < C::CH; ++c) v[(c * C::BOX_BYTES + keys * 128) / 16 + i] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (!(ok = warp_wait(&bar.p_full[g], pph, abort_flag, ws, 322))) break;
          pph ^= 1;
          tc_fence_after();
          if (lane == 0) {
            const uint64_t v0 = d_v + ((st * C::TILE_BYTES) >> 4);
            mma_ss(tm_o, v0, d_p, idesc, fresh);
            if (steps == 8) {
#pragma unroll
              for (int kk = 1; kk < 8; ++kk) mma_ss(tm_o, v0 + ((kk * 2048) >> 4), d_p + ((kk * 2048) >> 4), idesc, 1u);
            } else {
              for (int kk = 1; kk < steps; ++kk) mma_ss(tm_o, v0 + ((kk * 2048) >> 4), d_p + ((kk * 2048) >> 4), idesc, 1u);
            }
            mma_commit(&bar.empty[st]);
            mma_commit(&bar.p_empty[g]);
          }
          __syncwarp();
          fresh = 1;
        } else if (lane == 0) {
          mbar_arrive(&bar.empty[st]);
        }
        if (++st == C::STAGES) { st = C::KST; ph ^= 1; }
      }
      if (!ok) break;
      if (lane == 0) mma_commit(&bar.o_full[ob]);
      __syncwarp();
      if ((ob ^= 1) == 0) oph ^= 1;
    }
    if (lane == 0) {
      int never = 0;
      mma_commit(&bar.drain[1 + g]);
      mbar_wait(&bar.drain[1 + g], 0, &never, ws, 329);
    }
    __syncwarp();
  } else if (warp < C::EPI_WARPS) {
    // -------------------------------------------------------------- weights
    const int g = warp >> 2;                       // this group's blocks, S region and P buffer
    const int quad = warp & 3;
    const int key = (quad << 5) + lane;            // key within the block = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quad << 5) << 16;
    constexpr float scale_l2e = Scale<D>::value * kLog2e;
    uint8_t* prow = sP + g * C::P_BYTES + key * 128;
    uint32_t t = 0, sph = 0, pph = 0, rst = 0, rph = 0;
    float* my_log2n = s_log2n[warp];
    int* my_seen = s_seen[warp];
    const int token0 = lane / G, token1 = (lane + 32) / G;  // tokens of the columns this lane prepares
    bool ok = true;
    while (ok) {
      Segment seg;
      if (!(ok = seg_read<true>(bar.ring, rst, rph, &seg, abort_flag, ws, 330))) break;
      __syncwarp();
      seg_release(bar.ring, rst, rph, lane == 0);
      if (seg.j1 < 0) break;
      // N and log2 N of each row (column of S^T); rows past the last see nothing.
      const int rows = seg.m * G;
#pragma unroll
      for (int n = lane; n < NR; n += 32) {
        int seen = seg.n;
        if (a.causal) seen = max(0, min(seg.n, seg.n - seg.m + (n < 32 ? token0 : token1) + 1));
        my_seen[n] = n < rows ? seen : 0;
        my_log2n[n] = __log2f(static_cast<float>(max(seen, 1)));
      }
      const int least = a.causal ? max(0, seg.n - seg.m + 1) : seg.n;  // keys that every row sees
      __syncwarp();
      for (int j = seg.j0; j < seg.j1; ++j, ++t) {
        if ((t & 1) != static_cast<uint32_t>(g)) continue;
        if (!(ok = warp_wait(&bar.s_full[g], sph, abort_flag, ws, 331))) break;
        tc_fence_after();
        const bool cut = (j + 1) * kKeyBlock > least;
        const int at = j * kKeyBlock + key;
        // 32 columns at a time at most
        constexpr int W = NR < 32 ? NR : 32;
#pragma unroll
        for (int c0 = 0; c0 < NR; c0 += W) {
          uint32_t s[W];
          tmem_ld_cols(tmem + lane_off + C::TM_S + g * NR + c0, s);
          if (c0 + W == NR) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.s_empty[g]);
          }
          if (cut) {
#pragma unroll
            for (int n = 0; n < W; ++n)
              if (at >= my_seen[c0 + n]) s[n] = 0xff800000u;  // -inf: weight 0
          }
          // sigma(x) = 1 / (1 + 2^(log2 N - s scale log2 e)). Two MUFU operations
          // per weight, which this kernel's few weights allow. Relative error:
          // the exponent is an fp32 number, so log2 N and the sum are each off by
          // a few units in its last place (1e-6 at 1000 keys, 4e-6 at 2^24), the two
          // operations by 2e-7 each; the polynomial of the whole-sequence kernels
          // (sigmoid_n) spends 9e-4. The weight is then rounded to bf16 (2^-8 of it at
          // most), as in all forward kernels here: the second product's operands have one
          // type, V's. Against 64 bits the output is off by 0.0023 of its norm
          // that way, of which its own rounding alone is 0.0017.
#pragma unroll
          for (int n = 0; n < W; ++n)
            s[n] = __float_as_uint(rcp_approx(
                1.0f + ex2_approx(fmaf(__uint_as_float(s[n]), -scale_l2e, my_log2n[c0 + n]))));
          if (c0 == 0 && !(ok = warp_wait(&bar.p_empty[g], pph ^ 1, abort_flag, ws, 332))) break;
#pragma unroll
          for (int c = 0; c < W / 8; ++c) {
            const uint32_t* w = s + 8 * c;
            *reinterpret_cast<uint4*>(prow + (((c0 / 8 + c) ^ (key & 7)) << 4)) =
                make_uint4(pack_bf16x2(__uint_as_float(w[0]), __uint_as_float(w[1])),
                           pack_bf16x2(__uint_as_float(w[2]), __uint_as_float(w[3])),
                           pack_bf16x2(__uint_as_float(w[4]), __uint_as_float(w[5])),
                           pack_bf16x2(__uint_as_float(w[6]), __uint_as_float(w[7])));
          }
        }
        if (!ok) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[g]);
        sph ^= 1;
        pph ^= 1;
      }
    }
  } else {
    // --------------------------------------------------------------- output
    const int ow = warp - C::EPI_WARPS;            // lane quadrant
    const int dcol = (ow << 5) + lane;             // column of O = TMEM lane
    const bool mine = D == 128 || dcol < D;
    const uint32_t lane_off = static_cast<uint32_t>(ow << 5) << 16;
    uint32_t t = 0, ob = 0, oph = 0, rst = 0, rph = 0, parts = 0, red_ph = 0;
    bool ok = true;
    auto sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.joined);
      const bool done = warp_wait(&bar.joined, red_ph, abort_flag, ws, 336);
      red_ph ^= 1;
      return done;
    };
    // The sum of a tile's parts, by the output warps: `rows` rows of D, four at a
    // time. Lanes take four columns each, so a warp reads SUB rows of a part at
    // once; part p belongs to slice p % SLICES, the slices are added in order.
    // (Up to 16 parts, each thread adds its columns itself, eight loads at a time:
    // no exchange through shared memory.)
    auto join = [&](const Segment& seg, int rows) -> bool {
      constexpr int LPR = C::LPR, SLICES = C::SLICES, RC = C::RC, UNROLL = 3;
      const int np = seg.last_cta - seg.first_cta + 1;
      if (np <= 16) {
        for (int e = ow * 32 + lane; e < rows * LPR; e += C::OUT_WARPS * 32) {
          const float* part = a.parts + static_cast<size_t>(2 * seg.first_cta + 1) * (NR * D) + 4 * e;
          float4 sum = __ldcg(reinterpret_cast<const float4*>(part));
          part += NR * D;
#pragma unroll 1
          for (int p0 = 1; p0 < np; p0 += 8, part += 16 * (NR * D)) {
            float4 x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (p0 + u < np) x[u] = __ldcg(reinterpret_cast<const float4*>(part + 2 * u * (NR * D)));
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              sum.x += x[u].x;
              sum.y += x[u].y;
              sum.z += x[u].z;
              sum.w += x[u].w;
            }
          }
          const int n = e / LPR;
          *reinterpret_cast<uint2*>(a.o + (static_cast<size_t>(seg.start + n / G) * a.Hq + seg.head * G + n % G) * D +
                                    4 * (e % LPR)) = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
        }
        return true;
      }
      const int slice = ow * C::SUB + lane / LPR, l4 = lane % LPR;
      float4* red = reinterpret_cast<float4*>(smem + C::OFF_RED);
      for (int n0 = 0; n0 < rows; n0 += RC) {
        float4 sum[RC];
#pragma unroll
        for (int i = 0; i < RC; ++i) sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = slice; p0 < np; p0 += SLICES * UNROLL) {
          float4 x[UNROLL][RC];
#pragma unroll
          for (int u = 0; u < UNROLL; ++u) {
            // the first part lies in its CTA's second place, the others in their CTA's first
            const int p = p0 + u * SLICES;
            const float* part = a.parts + static_cast<size_t>(2 * (seg.first_cta + p) + (p == 0)) * (NR * D) + 4 * l4;
#pragma unroll
            for (int i = 0; i < RC; ++i) {
              x[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (p < np && n0 + i < rows) x[u][i] = __ldcg(reinterpret_cast<const float4*>(part + (n0 + i) * D));
            }
          }
#pragma unroll
          for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int i = 0; i < RC; ++i) {
              sum[i].x += x[u][i].x;
              sum[i].y += x[u][i].y;
              sum[i].z += x[u][i].z;
              sum[i].w += x[u][i].w;
            }
        }
#pragma unroll
        for (int i = 0; i < RC; ++i) red[(slice * RC + i) * LPR + l4] = sum[i];
        if (!sync()) return false;
        for (int pair = ow * 32 + lane; pair < RC * D / 2; pair += C::OUT_WARPS * 32) {
          const int n = n0 + pair / (D / 2), c = pair % (D / 2);
          if (n >= rows) break;
          float2 s = make_float2(0.f, 0.f);
          const float2* from = reinterpret_cast<const float2*>(red) + pair;
          for (int k = 0; k < min(np, SLICES); ++k) {
            const float2 x = from[k * RC * (D / 2)];
            s.x += x.x;
            s.y += x.y;
          }
          reinterpret_cast<uint32_t*>(
              a.o + (static_cast<size_t>(seg.start + n / G) * a.Hq + seg.head * G + n % G) * D)[c] = pack_bf16x2(s.x, s.y);
        }
        if (!sync()) return false;
      }
      return true;
    };
    while (ok) {
      Segment seg;
      if (!(ok = seg_read<true>(bar.ring, rst, rph, &seg, abort_flag, ws, 340))) break;
      __syncwarp();
      seg_release(bar.ring, rst, rph, lane == 0);
      if (seg.j1 < 0) break;
      const int rows = seg.m * G, len = seg.j1 - seg.j0;
      // Which groups had blocks of this segment.
      const bool both = len > 1;
      const uint32_t only = t & 1;
      t += len;
      if (!(ok = warp_wait(&bar.o_full[ob], oph, abort_flag, ws, 333))) break;
      tc_fence_after();
      const bool whole = len == seg.blocks;
      __nv_bfloat16* dst = a.o + (static_cast<size_t>(seg.start) * a.Hq + seg.head * G) * D + dcol;
      float* part = a.parts + static_cast<size_t>(2 * blockIdx.x + (seg.j0 == 0)) * (NR * D) + dcol;
      int head = 0;
#pragma unroll
      for (int c = 0; c < NR / 16; ++c) {
        if (16 * c >= rows) break;
        uint32_t x[16];
        const uint32_t from = tmem + lane_off + C::TM_O + 2 * ob * NR + 16 * c;
        tmem_ld16(from + (both ? 0 : only * NR), x);
        if (both) {
          uint32_t y[16];
          tmem_ld16(from + NR, y);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) + __uint_as_float(y[i]));
        }
        if (!mine) continue;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (16 * c + i >= rows) break;
          if (whole) {
            *dst = __float2bfloat16(__uint_as_float(x[i]));
            dst += D;
            if (++head == G) {  // on to the next token's first head
              head = 0;
              dst += static_cast<size_t>(a.Hq - G) * D;
            }
          } else {
            __stcg(part + (16 * c + i) * D, __uint_as_float(x[i]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.o_empty[ob]);
      if ((ob ^= 1) == 0) oph ^= 1;
      if (whole) continue;
      if (!(ok = last_part(&bar.stored, &bar.counted, &bar.last, seg, ws, ow, lane, parts, abort_flag, 334))) break;
      parts ^= 1;
      if (bar.last && !(ok = join(seg, rows))) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kIssueO) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

namespace {

template <int D, int NR, typename U>
cudaError_t launch_few_impl(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttend& a,
                            int grid, cudaStream_t stream) {
  using C = FewCfg<D, NR>;
  static PerDeviceOnce attr;
  const cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(paged_few_kernel<D, NR, U>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
  });
  if (e != cudaSuccess) return e;
  return launch_programmatic(paged_few_kernel<D, NR, U>, dim3(grid), dim3(C::THREADS), C::SMEM_ALLOC, stream, tq, tk, tv,
                             a);
}

template <typename U, typename... Args>
cudaError_t launch_few(int d, int rows, Args&&... args) {
  if (d == 64) {
    if (rows <= 16) return launch_few_impl<64, 16, U>(args...);
    if (rows <= 32) return launch_few_impl<64, 32, U>(args...);
    return launch_few_impl<64, 64, U>(args...);
  }
  if (rows <= 16) return launch_few_impl<128, 16, U>(args...);
  return launch_few_impl<128, 32, U>(args...);
}

}  // namespace

cudaError_t launch_paged_few(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttend& a,
                             bool wide, int grid, cudaStream_t stream) {
  const int rows = a.max_q * (a.Hq / a.Hkv);
  return wide ? launch_few<unsigned long long>(a.d, rows, tq, tk, tv, a, grid, stream)
              : launch_few<uint32_t>(a.d, rows, tq, tk, tv, a, grid, stream);
}

}  // namespace sigattn
