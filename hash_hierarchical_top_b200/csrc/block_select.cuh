// Block selection for grouped-query attention: each query of a chunk chooses, per KV group (or
// query head), the blocks whose mean key scores highest with its summed heads.
//
//   score[p] = (sum_h q_h) . mean_p over the row's heads, rounded to fp32 once;
//
// The products and sums are in 64 bits: bf16 x fp32 products are exact there and a sum of 128 of
// them is off by 2^-45 of its terms at most, so the rounded score does not depend on the order
// of the sum and the chosen set is that of the definition. The m largest are kept, ties to the
// lower block.
#pragma once
#include "common.cuh"
#include "select.cuh"

namespace hhr {

struct BlockSelectArgs {
  const uint16_t* q;         // [B][T][Hq][d]
  const int32_t* seq_len;
  const int32_t* q_pos;      // [B][T] or null
  const int32_t* page_table;
  const float* block_mean;   // [n_phys][G][d]
  float* scores;             // [B][T][Gs][maxp]
  int32_t* out;              // [B][T][Gs][m_max]
  int32_t* out_count;        // [B][T][Gs]
  int B, T, Hq, G, Gs, kv_div, P, maxp, n_phys, m_pages, m_max, sink, local;
};

constexpr int kBsPages = 32;    // blocks per CTA
constexpr int kBsQueries = 8;   // rows at a time
constexpr int kBsThreads = 256;

// Blocks that the query (b, t) may choose: those that begin at or before its position.
__device__ __forceinline__ int eligible_blocks(const BlockSelectArgs& a, int b, int t) {
  int n = min(max(a.seq_len[b], 0), a.maxp * a.P);
  if (a.q_pos != nullptr) n = min(n - 1, a.q_pos[(size_t)b * a.T + t]) + 1;
  return ceil_div(max(n, 0), a.P);
}

// Grid (block tile, KV group, sequence): the tile's means are staged once and scored against
// every row of the group, kBsQueries rows at a time: warp w takes row w, lane l block l.
__global__ void __launch_bounds__(kBsThreads) block_mean_score_kernel(BlockSelectArgs a) {
  __shared__ __align__(16) float mean[kBsPages][kD + 4];
  __shared__ __align__(16) double qs[kBsQueries][kD];
  const int b = blockIdx.z, g = blockIdx.y, p0 = blockIdx.x * kBsPages, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int n_b = ceil_div(min(max(a.seq_len[b], 0), a.maxp * a.P), a.P);
  if (p0 >= n_b) return;
  for (int i = tid; i < kBsPages * (kD / 4); i += kBsThreads) {
    const int p = i / (kD / 4), c = i % (kD / 4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p0 + p < n_b) {
      const int phys = a.page_table[(size_t)b * a.maxp + p0 + p];
      if (phys >= 0 && phys < a.n_phys)
        v = reinterpret_cast<const float4*>(a.block_mean + ((size_t)phys * a.G + g) * kD)[c];
      else
        v.x = __int_as_float(0x7fffffff);  // NaN: a block without a page is never chosen
      if (c == 0 && (phys < 0 || phys >= a.n_phys)) flag_status(kStatusBadPage);
    }
    *reinterpret_cast<float4*>(&mean[p][4 * c]) = v;
  }
  const int gs = a.Hq / a.Gs, rows = a.T * a.kv_div;  // rows of this KV group: (t, j)
  for (int r0 = 0; r0 < rows; r0 += kBsQueries) {
    __syncthreads();
    for (int i = tid; i < kBsQueries * kD; i += kBsThreads) {
      const int r = r0 + i / kD, c = i % kD;
      double s = 0.0;
      if (r < rows) {
        const int t = r / a.kv_div, j = r % a.kv_div;
        const uint16_t* q = a.q + (((size_t)b * a.T + t) * a.Hq + (size_t)(g * a.kv_div + j) * gs) * kD + c;
        for (int h = 0; h < gs; ++h) s += (double)bf16_to_f(q[(size_t)h * kD]);
      }
      qs[i / kD][c] = s;
    }
    __syncthreads();
    const int r = r0 + warp;
    if (r >= rows) continue;
    const int t = r / a.kv_div, j = r % a.kv_div;
    double s0 = 0.0, s1 = 0.0, s2 = 0.0, s3 = 0.0;
#pragma unroll 8
    for (int c = 0; c < kD; c += 4) {
      const float4 m = *reinterpret_cast<const float4*>(&mean[lane][c]);
      s0 = fma(qs[warp][c], (double)m.x, s0);
      s1 = fma(qs[warp][c + 1], (double)m.y, s1);
      s2 = fma(qs[warp][c + 2], (double)m.z, s2);
      s3 = fma(qs[warp][c + 3], (double)m.w, s3);
    }
    const size_t row = ((size_t)b * a.T + t) * a.Gs + g * a.kv_div + j;
    // + 0: a score of -0 ties with +0.
    if (p0 + lane < n_b) a.scores[row * a.maxp + p0 + lane] = (float)((s0 + s1) + (s2 + s3)) + 0.f;
  }
}

// One CTA per row: the m largest scores of its eligible blocks, in ascending block order.
constexpr int kBsSelThreads = 512;
__global__ void __launch_bounds__(kBsSelThreads) block_topm_kernel(BlockSelectArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ SelShared<4> sh;
  extern __shared__ uint32_t bs_keys[];
  const int row = blockIdx.x, tid = threadIdx.x;
  const int bt = row / a.Gs, b = bt / a.T;
  const int n = eligible_blocks(a, b, bt - b * a.T);
  int32_t* out = a.out + (size_t)row * a.m_max;
  const int k = block_select_largest<kBsSelThreads, kSelLoadUnroll, 4>(
      a.scores + (size_t)row * a.maxp, n, bs_keys, sh, true, a.m_pages, 0, 0, out, a.m_max, nullptr,
      0, a.sink, a.local);
  for (int i = k + tid; i < a.m_max; i += kBsSelThreads) out[i] = -1;
  if (tid == 0) a.out_count[row] = k;
}

}  // namespace hhr
