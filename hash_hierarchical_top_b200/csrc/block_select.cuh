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

// Blocks that the query (b, t) may choose: those that begin at or before its position.
__device__ __forceinline__ int eligible_blocks(const BlockSelectArgs& a, int b, int t) {
  int n = min(max(a.seq_len[b], 0), a.maxp * a.P);
  if (a.q_pos != nullptr) n = min(n - 1, a.q_pos[(size_t)b * a.T + t]) + 1;
  return ceil_div(max(n, 0), a.P);
}

// Rows of a KV group over the chunk, r = t kv_div + j: row (b, t, g kv_div + j).
__device__ __forceinline__ size_t bs_row(const BlockSelectArgs& a, int b, int g, int r) {
  const int t = r / a.kv_div, j = r - t * a.kv_div;
  return ((size_t)b * a.T + t) * a.Gs + (size_t)g * a.kv_div + j;
}
// First query channel of such a row.
__device__ __forceinline__ const uint16_t* bs_query(const BlockSelectArgs& a, size_t row) {
  const size_t bt = row / a.Gs;
  return a.q + (bt * a.Hq + (row - bt * a.Gs) * (a.Hq / a.Gs)) * kD;
}
// Physical page of block p of sequence b, or -1 with the status word set (such a block scores
// NaN: it is never chosen).
__device__ __forceinline__ int bs_page(const BlockSelectArgs& a, int b, int p) {
  const int phys = a.page_table[(size_t)b * a.maxp + p];
  if (phys >= 0 && phys < a.n_phys) return phys;
  flag_status(kStatusBadPage);
  return -1;
}
__device__ __forceinline__ double shfl_xor_f64(double v, int o) {
  return __hiloint2double(__shfl_xor_sync(kFull, __double2hiint(v), o),
                          __shfl_xor_sync(kFull, __double2loint(v), o));
}
// A score as it is kept: rounded once; + 0 so that -0 ties with +0.
__device__ __forceinline__ float bs_round(double s) { return (float)s + 0.f; }

// One row per KV group (single tokens): a stream over the means, 512 B per block. A warp takes
// 32 blocks, a lane 4 channels of each; 8 blocks' loads are in flight per warp, and a transposed
// reduction leaves block l's sum on lane l (31 exchanges for 32 sums). Grid (blocks / 128, KV
// group, sequence).
constexpr int kBvWarps = 4;
__global__ void __launch_bounds__(kBvWarps * 32, 4) block_mean_stream_kernel(BlockSelectArgs a) {
  const int b = blockIdx.z, g = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int p0 = (blockIdx.x * kBvWarps + warp) * 32;
  const int n_b = ceil_div(min(max(a.seq_len[b], 0), a.maxp * a.P), a.P);
  if (p0 >= n_b) return;
  const int mine = p0 + lane < n_b ? bs_page(a, b, p0 + lane) : -1;
  const size_t row = bs_row(a, b, g, 0);
  double q[4] = {0.0, 0.0, 0.0, 0.0};
  {
    const uint16_t* qp = bs_query(a, row) + 4 * lane;
    for (int h = 0; h < a.Hq / a.Gs; ++h) {
      const float4 f = bf16x4_to_f4(*reinterpret_cast<const uint2*>(qp + (size_t)h * kD));
      q[0] += (double)f.x; q[1] += (double)f.y; q[2] += (double)f.z; q[3] += (double)f.w;
    }
  }
  double v[32];
#pragma unroll
  for (int i0 = 0; i0 < 32; i0 += 8) {
    float4 m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int phys = __shfl_sync(kFull, mine, i0 + i);
      m[i] = phys >= 0 ? ldg_f4_now(reinterpret_cast<const float4*>(
                             a.block_mean + ((size_t)phys * a.G + g) * kD) + lane)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i0 + i] = fma(q[0], (double)m[i].x, fma(q[1], (double)m[i].y,
                  fma(q[2], (double)m[i].z, q[3] * (double)m[i].w)));
  }
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) {
    const bool upper = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const double send = upper ? v[i] : v[i + s], keep = upper ? v[i + s] : v[i];
      v[i] = keep + shfl_xor_f64(send, s);
    }
  }
  if (p0 + lane < n_b)
    a.scores[row * a.maxp + p0 + lane] = mine >= 0 ? bs_round(v[0]) : __int_as_float(0x7fffffff);
}

// Several rows per KV group (a chunk of queries, or a row per head): a tile of kBtPages blocks
// by kBtRows rows in 64 bits, both operands staged in shared memory once as doubles (so each is
// converted once per tile); a thread sums 2 blocks x 4 rows, reading two channels at a time.
// Grid (block tile, KV group x row tile, sequence).
constexpr int kBtPages = 32, kBtRows = 64, kBtThreads = 256;
constexpr int kBtStride = kD + 2;  // doubles; 16-byte rows, and rows 4 banks apart
inline size_t block_tile_smem() { return (size_t)(kBtPages + kBtRows) * kBtStride * 8; }
__global__ void __launch_bounds__(kBtThreads) block_mean_tile_kernel(BlockSelectArgs a) {
  extern __shared__ double bt_smem[];
  double* ms = bt_smem;                        // [kBtPages][kBtStride]
  double* qs = bt_smem + kBtPages * kBtStride; // [kBtRows][kBtStride]
  const int b = blockIdx.z, p0 = blockIdx.x * kBtPages, tid = threadIdx.x;
  const int g = blockIdx.y % a.G, r0 = (blockIdx.y / a.G) * kBtRows;
  const int n_b = ceil_div(min(max(a.seq_len[b], 0), a.maxp * a.P), a.P);
  if (p0 >= n_b) return;
  const int rows = min(kBtRows, a.T * a.kv_div - r0);
  for (int i = tid; i < kBtPages * (kD / 4); i += kBtThreads) {
    const int p = i / (kD / 4), c = 4 * (i % (kD / 4));
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p0 + p < n_b) {
      const int phys = bs_page(a, b, p0 + p);
      if (phys >= 0)
        f = *reinterpret_cast<const float4*>(a.block_mean + ((size_t)phys * a.G + g) * kD + c);
      else
        f.x = __int_as_float(0x7fffffff);
    }
    double2* d = reinterpret_cast<double2*>(ms + p * kBtStride + c);
    d[0] = make_double2(f.x, f.y);
    d[1] = make_double2(f.z, f.w);
  }
  const int gs = a.Hq / a.Gs;
  for (int i = tid; i < kBtRows * (kD / 4); i += kBtThreads) {
    const int r = i / (kD / 4), c = 4 * (i % (kD / 4));
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    if (r < rows) {
      const uint16_t* qp = bs_query(a, bs_row(a, b, g, r0 + r)) + c;
      for (int h = 0; h < gs; ++h) {
        const float4 f = bf16x4_to_f4(*reinterpret_cast<const uint2*>(qp + (size_t)h * kD));
        s[0] += (double)f.x; s[1] += (double)f.y; s[2] += (double)f.z; s[3] += (double)f.w;
      }
    }
    double2* d = reinterpret_cast<double2*>(qs + r * kBtStride + c);
    d[0] = make_double2(s[0], s[1]);
    d[1] = make_double2(s[2], s[3]);
  }
  __syncthreads();
  // Threads 16 x 16: blocks tx, tx + 16; rows ty + 16 k.
  const int tx = tid & 15, ty = tid >> 4;
  double acc[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k][0] = acc[k][1] = 0.0;
  const int nk = (rows - ty + 15) / 16;  // rows of this thread
#pragma unroll 4
  for (int c = 0; c < kD; c += 2) {
    const double2 m0 = *reinterpret_cast<const double2*>(ms + tx * kBtStride + c);
    const double2 m1 = *reinterpret_cast<const double2*>(ms + (tx + 16) * kBtStride + c);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k < nk) {
        const double2 q = *reinterpret_cast<const double2*>(qs + (ty + 16 * k) * kBtStride + c);
        acc[k][0] = fma(q.x, m0.x, acc[k][0]);
        acc[k][1] = fma(q.x, m1.x, acc[k][1]);
        acc[k][0] = fma(q.y, m0.y, acc[k][0]);
        acc[k][1] = fma(q.y, m1.y, acc[k][1]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k >= nk) break;
    float* out = a.scores + bs_row(a, b, g, r0 + ty + 16 * k) * a.maxp + p0;
    if (p0 + tx < n_b) out[tx] = bs_round(acc[k][0]);
    if (p0 + tx + 16 < n_b) out[tx + 16] = bs_round(acc[k][1]);
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
