// paged.cu -- sigmoid attention of a chunk of new tokens over a paged cache.
//
//   o_i = sum_{j < N} sigma(q_i . k_j / sqrt(d) - ln N) v_j
//
// One warp per (row, query head): each lane takes one key of 32 for the
// scores, then d / 32 columns of V for the sums.
#include "paged.cuh"

namespace sigattn {

template <int D>
__global__ void __launch_bounds__(256) paged_rows_kernel(PagedAttend a) {
  grid_dep_launch();
  grid_dep_wait();
  constexpr int C = D / 32;
  __shared__ float sq[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long units = static_cast<long long>(a.total) * a.Hq;
  const int G = a.Hq / a.Hkv, most = a.max_pages << a.page_shift, ps = 1 << a.page_shift;
  for (int b = blockIdx.x * 256 + threadIdx.x; b < a.B; b += gridDim.x * 256) {
    const int s = a.cu[b], e = a.cu[b + 1], n = a.kv[b];
    if (s < 0 || e < s || e > a.total || e - s > a.max_q || n < 0 || n > most) raise_invalid(a.ws, -(b + 1));
  }
  for (long long u = blockIdx.x * 8LL + warp; u < units; u += gridDim.x * 8LL) {
    const int t = static_cast<int>(u / a.Hq), h = static_cast<int>(u % a.Hq);
    int seq = -1, start = 0, end = 0, n = 0;
    for (int b = lane; b < a.B; b += 32) {
      const int s = a.cu[b], e = a.cu[b + 1], nb = a.kv[b];
      if (s < 0 || e < s || e > a.total || e - s > a.max_q || nb < 0 || nb > most) continue;
      if (s <= t && t < e) seq = b;
    }
    const unsigned found = __ballot_sync(0xffffffffu, seq >= 0);
    if (found == 0) continue;
    seq = __shfl_sync(0xffffffffu, seq, __ffs(found) - 1);
    start = a.cu[seq];
    end = a.cu[seq + 1];
    n = a.kv[seq];
    int seen = n;
    if (a.causal) seen = min(n, max(0, n - (end - start) + (t - start) + 1));
    for (int c = lane; c < D; c += 32)
      sq[warp][c] = __bfloat162float(a.q[t * a.q_stride + h * D + c]) * Scale<D>::value;
    __syncwarp();
    float acc[C] = {};
    const float bias = -logf(static_cast<float>(max(seen, 1)));
    for (int j0 = 0; j0 < seen; j0 += 32) {
      const int j = j0 + lane;
      float p = 0.f;
      size_t row = 0;
      int page = -1;
      if (j < seen) {
        page = a.table[static_cast<size_t>(seq) * a.max_pages + (j >> a.page_shift)];
        if (page < 0 || page >= a.num_pages) {
          raise_invalid(a.ws, 203);
          page = -1;
        }
      }
      if (page >= 0) {
        row = ((static_cast<size_t>(page) * a.Hkv + h / G) << a.page_shift) + (j & (ps - 1));
        const uint4* kr = reinterpret_cast<const uint4*>(a.k_cache + row * D);
        float s = 0.f;
        for (int c = 0; c < D / 8; ++c) {
          const uint4 w = kr[c];
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
          for (int e = 0; e < 4; ++e)
            s += __uint_as_float(ww[e] << 16) * sq[warp][8 * c + 2 * e] +
                 __uint_as_float(ww[e] & 0xffff0000u) * sq[warp][8 * c + 2 * e + 1];
        }
        p = 1.0f / (1.0f + expf(-(s + bias)));
      }
      for (int l = 0; l < 32; ++l) {
        const float pl = __shfl_sync(0xffffffffu, p, l);
        const unsigned long long rl = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(row), l);
        if (__shfl_sync(0xffffffffu, page, l) < 0) continue;
        for (int c = 0; c < C; ++c) acc[c] += pl * __bfloat162float(a.v_cache[rl * D + c * 32 + lane]);
      }
    }
    for (int c = 0; c < C; ++c)
      a.o[(static_cast<size_t>(t) * a.Hq + h) * D + c * 32 + lane] = __float2bfloat16(acc[c]);
    __syncwarp();
  }
}

cudaError_t launch_fwd_paged(const PagedAttend& a, int num_sms, cudaStream_t stream) {
  const int grid = static_cast<int>(std::max(
      1LL, std::min(8LL * num_sms, (static_cast<long long>(a.total) * a.Hq + 7) / 8)));
  return launch_programmatic(a.d == 64 ? paged_rows_kernel<64> : paged_rows_kernel<128>, dim3(grid), dim3(256), 0,
                             stream, a);
}

}  // namespace sigattn
