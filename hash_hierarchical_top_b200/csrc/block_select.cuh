// Block selection for grouped-query attention: each query of a chunk chooses, per KV group (or
// query head), the blocks whose mean key scores highest with its summed heads.
//
//   score[p] = (sum_h q_h) . mean_p over the row's heads, the 64-bit sum rounded to fp32 once;
//   the m largest are kept, ties to the lower block.
//
// The scores are computed in fp32 with a bound on their error, which settles all blocks but
// those near the cut: with |s - score| <= E for every block of a row, the m-th largest score is
// within E of the m-th largest s (tau), so a block with s > tau + 2E is kept and one with
// s < tau - 2E is not. The blocks in between (nearly always the cut itself, alone) are scored
// again in 64 bits, where bf16 x fp32 products are exact and 128 of them sum to 2^-45 of their
// size. Scoring everything in 64 bits took 22.7 us where the fp32 tiles take 11.4 (64 queries x 8
// groups over 1024 blocks, cold caches); the single-token stream takes 28 us either way.
//
// Measured (calls in a row): 8 sequences of 4096 blocks x 8 groups, one token each, 37 us: a stream
// of 134 MB (20.5 us at the copy rate; 27.5 us with its launch and the three dependent loads that
// precede the first means) and a choice that is a chain of barriers on 64 CTAs (about 6 us); 64
// queries over 1024 blocks 17.8 us, all latency.
//
// E = kBsErr ||A|| max_p ||mean_p||, A_c = sum_h |q_hc|: the fp32 sum over at most 8 heads is off
// by 7 units of 2^-24 of A_c, products and sums over 128 channels by at most 16 + 8 (chains of
// 16, then at most 8 additions), the norms themselves by a few 2^-24 of the whole.
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
  float* norms;              // [B][G][maxp] squares of the means' norms
  int32_t* out;              // [B][T][Gs][m_max]
  int32_t* out_count;        // [B][T][Gs]
  int B, T, Hq, G, Gs, kv_div, P, maxp, n_phys, m_pages, m_max, sink, local;
  uint32_t g_mul;            // ceil(2^32 / G): i / G = umulhi(i, g_mul) for 1 < G <= 64, i < 2^26
};

// Blocks that the query (b, t) may choose: those that begin at or before its position.
__device__ __forceinline__ int eligible_blocks(const BlockSelectArgs& a, int b, int t) {
  int n = min(max(a.seq_len[b], 0), a.maxp * a.P);
  if (a.q_pos != nullptr) n = min(n - 1, a.q_pos[(size_t)b * a.T + t]) + 1;
  return ceil_div(max(n, 0), a.P);
}

// Row of a KV group over the chunk, r = t kv_div + j: row (b, t, g kv_div + j), and its first
// query channel. (32-bit divisions: a 64-bit one costs as much as a row's arithmetic.)
__device__ __forceinline__ size_t bs_row(const BlockSelectArgs& a, int b, int g, int r) {
  const int t = a.kv_div == 1 ? r : r / a.kv_div, j = r - t * a.kv_div;
  return ((size_t)b * a.T + t) * a.Gs + (size_t)g * a.kv_div + j;
}
// First channel of query row r of sequence b and KV group g.
__device__ __forceinline__ const uint16_t* bs_query(const BlockSelectArgs& a, int b, int g, int r) {
  const int t = a.kv_div == 1 ? r : r / a.kv_div, j = r - t * a.kv_div;
  const int gs = a.Hq / a.Gs;
  return a.q + (((size_t)b * a.T + t) * a.Hq + (size_t)(g * a.kv_div + j) * gs) * kD;
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
// Four channels of a row's query over its gs <= NH heads, loaded at once: absent heads are read
// as the last one (a conditional load would keep the next one waiting) and not used.
template <int NH>
__device__ __forceinline__ void bs_heads(const uint16_t* q, int gs, uint2 (&w)[NH]) {
#pragma unroll
  for (int h = 0; h < NH; ++h) w[h] = *reinterpret_cast<const uint2*>(q + (size_t)min(h, gs - 1) * kD);
}
// Their sums, in 64 bits (exact but for the last of 53) and in fp32.
__device__ __forceinline__ void bs_query_sum(const uint16_t* q, int gs, double (&s)[4]) {
  uint2 w[kMaxGroup];
  bs_heads<kMaxGroup>(q, gs, w);
  s[0] = s[1] = s[2] = s[3] = 0.0;
#pragma unroll
  for (int h = 0; h < kMaxGroup; ++h) {
    if (h < gs) {
      const float4 f = bf16x4_to_f4(w[h]);
      s[0] += (double)f.x; s[1] += (double)f.y; s[2] += (double)f.z; s[3] += (double)f.w;
    }
  }
}
template <int NH>
__device__ __forceinline__ float4 bs_query_sum_f32(const uint16_t* q, int gs) {
  uint2 w[NH];
  bs_heads<NH>(q, gs, w);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    const float4 f = bf16x4_to_f4(h < gs ? w[h] : make_uint2(0u, 0u));
    s.x += f.x; s.y += f.y; s.z += f.z; s.w += f.w;
  }
  return s;
}
// A score as it is kept; + 0 so that -0 ties with +0.
__device__ __forceinline__ float bs_round(double s) { return (float)s + 0.f; }
// The definition's score of block p with a row's query sums (channels 4 lane + {0..3}); a warp.
__device__ __forceinline__ float bs_exact(const BlockSelectArgs& a, int b, int g, int p,
                                          const double (&q)[4], int lane) {
  const int phys = bs_page(a, b, p);
  if (phys < 0) return __int_as_float(0x7fffffff);
  const float4 m =
      reinterpret_cast<const float4*>(a.block_mean + ((size_t)phys * a.G + g) * kD)[lane];
  double s = fma(q[0], (double)m.x, fma(q[1], (double)m.y, fma(q[2], (double)m.z, q[3] * (double)m.w)));
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += shfl_xor_f64(s, o);
  return bs_round(s);
}
constexpr float kBsErr = 40.f * 5.9604645e-08f;  // 40 * 2^-24

// Blocks of sequence b that hold keys.
__device__ __forceinline__ int bs_blocks(const BlockSelectArgs& a, int b) {
  return ceil_div(min(max(a.seq_len[b], 0), a.maxp * a.P), a.P);
}

// One row per KV group (single tokens): a stream over the means. The means of a page's KV groups
// lie side by side (512 G bytes), so the rows of a sequence are taken in the order (page, group),
// as they lie in memory. The pages of all sequences are laid end to end and divided evenly over a grid
// that fills the GPU; warp w of a CTA takes the rows 16 w .. 16 w + 15, then those 64 on. 8 lanes
// share a row, in registers: as soon as a row has been multiplied, its registers take the row of
// the same place in the warp's next item (8 KB in flight per warp).
constexpr int kBvWarps = 4;
constexpr int kBvCtasPerSm = 3;  // 4 spill, and are no faster
constexpr int kBvItem = 16;      // rows of an item
constexpr int kBvMaxGroups = 64; // KV groups whose query sums are staged
inline size_t block_stream_smem(int G) { return (size_t)G * kD * 4; }
__global__ void __launch_bounds__(kBvWarps * 32, kBvCtasPerSm)
    block_mean_stream_kernel(BlockSelectArgs a) {
  extern __shared__ __align__(16) float bv_q[];  // [G][d] query sums of the sequence
  __shared__ int sh[40];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lg = lane >> 3, lc = lane & 7;  // row of a step, channel part
  constexpr int NK = kBvItem / 4;
  pdl_wait();
  pdl_trigger();
  const UnitPlace at = place_units(a.B, sh, [&](int b) { return bs_blocks(a, b); }, [&](int all) {
    return all == 0 ? -1 : min(share_begin(blockIdx.x, all, gridDim.x), all - 1);
  });
  int left = share_begin(blockIdx.x, at.total, gridDim.x);
  int p0 = left - at.before;
  left = share_begin(blockIdx.x + 1, at.total, gridDim.x) - left;
  for (int b = at.b; left > 0; ++b, p0 = 0) {
    const int n_b = bs_blocks(a, b), p1 = min(n_b, p0 + left);
    if (p1 <= p0) continue;
    left -= p1 - p0;
    const int end = p1 * a.G;  // rows (page, group) [p0 G, end) of the sequence
    const int32_t* pages = a.page_table + (size_t)b * a.maxp;
    // Lane l < 16 locates row l of an item: its page-table entry (left alone for an item after it
    // is loaded: a use at once would stall the warp for the load's latency), then its row of the
    // means. kNone: past the end.
    constexpr int kNone = (int)0x80000000;
    auto page_of_row = [&](int i) { return a.G == 1 ? i : (int)__umulhi((uint32_t)i, a.g_mul); };
    auto page_at = [&](int i) { return lane < kBvItem && i < end ? pages[page_of_row(i)] : kNone; };
    auto row_at = [&](int i, int page) {
      if (page >= 0 && page < a.n_phys) return page * a.G + (i - page_of_row(i) * a.G);
      if (page != kNone) flag_status(kStatusBadPage);
      return -1;
    };
    float4 f[NK][4];  // row 4 k + lg, channels 32 i + 4 lc + {0..3}
    auto load = [&](int rows, int k) {
      const int r = __shfl_sync(kFull, rows, 4 * k + lg);
      const float4* m4 = reinterpret_cast<const float4*>(a.block_mean + (size_t)max(r, 0) * kD) + lc;
#pragma unroll
      for (int i = 0; i < 4; ++i) f[k][i] = ldg_f4_now(m4 + 8 * i);  // no such row: not used
    };
    int i0 = p0 * a.G + warp * kBvItem;  // first row of the item
    constexpr int kStep = kBvWarps * kBvItem;
    int pg = page_at(i0 + lane), pg_next = page_at(i0 + kStep + lane);
    int rows = row_at(i0 + lane, pg);
#pragma unroll
    for (int k = 0; k < NK; ++k) load(rows, k);
    __syncthreads();  // the previous sequence's query sums have been used
    for (int i = tid; i < a.G * (kD / 4); i += kBvWarps * 32) {
      const int g = i / (kD / 4), c = i % (kD / 4);
      reinterpret_cast<float4*>(bv_q)[i] =
          bs_query_sum_f32<kMaxGroup>(bs_query(a, b, g, 0) + 4 * c, a.Hq / a.Gs);
    }
    __syncthreads();
    for (; i0 < end; i0 += kStep) {
      const int rows_next = row_at(i0 + kStep + lane, pg_next);
      pg_next = page_at(i0 + 2 * kStep + lane);
      float v[NK], u[NK];  // score and square norm of the step's row
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const int i = min(i0 + 4 * k + lg, end - 1);
        const int g = i - page_of_row(i) * a.G;
        const float4* q4 = reinterpret_cast<const float4*>(bv_q + g * kD) + lc;
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 q = q4[8 * j], m = f[k][j];
          x = fmaf(q.x, m.x, x);
          x = fmaf(q.y, m.y, x);
          x = fmaf(q.z, m.z, x);
          x = fmaf(q.w, m.w, x);
          y = fmaf(m.x, m.x, y);
          y = fmaf(m.y, m.y, y);
          y = fmaf(m.z, m.z, y);
          y = fmaf(m.w, m.w, y);
        }
        v[k] = x;
        u[k] = y;
        load(rows_next, k);
      }
      // Over the 8 lanes of a row: v[0] of lane lc ends as the sum of step lc / 2.
#pragma unroll
      for (int o = 4, w = NK / 2; w >= 1; o >>= 1, w >>= 1) {
        const bool upper = (lc & o) != 0;
#pragma unroll
        for (int k = 0; k < w; ++k) {
          const float sv = upper ? v[k] : v[k + w], kv = upper ? v[k + w] : v[k];
          v[k] = kv + __shfl_xor_sync(kFull, sv, o);
          const float su = upper ? u[k] : u[k + w], ku = upper ? u[k + w] : u[k];
          u[k] = ku + __shfl_xor_sync(kFull, su, o);
        }
      }
      v[0] += __shfl_xor_sync(kFull, v[0], 1);
      u[0] += __shfl_xor_sync(kFull, u[0], 1);
      const int j = 4 * (lc >> 1) + lg, i = i0 + j;
      const bool held = __shfl_sync(kFull, rows, j) >= 0;
      if ((lc & 1) == 0 && i < end) {
        const int p = page_of_row(i);
        const size_t o = ((size_t)b * a.G + (i - p * a.G)) * a.maxp + p;
        a.scores[o] = held ? v[0] + 0.f : __int_as_float(0x7fffffff);
        a.norms[o] = held ? u[0] : __int_as_float(0x7fffffff);
      }
      rows = rows_next;
    }
  }
}

// Several rows per KV group (a chunk of queries, or a row per head): a tile of kBtPages blocks
// by kBtRows rows, both staged in shared memory; a thread sums 2 blocks x 4 rows, 16 channels at
// a time. Grid (block tile, KV group x row tile, sequence).
constexpr int kBtPages = 32, kBtRows = 32, kBtThreads = 128;
constexpr int kBtStride = kD + 4;  // 16-byte rows, 4 banks apart
inline size_t block_tile_smem() { return (size_t)(kBtPages + kBtRows) * kBtStride * 4; }
template <int NH>
__global__ void __launch_bounds__(kBtThreads, 4) block_mean_tile_kernel(BlockSelectArgs a) {
  extern __shared__ __align__(16) float bt_smem[];
  float* ms = bt_smem;                         // [kBtPages][kBtStride]
  float* qs = bt_smem + kBtPages * kBtStride;  // [kBtRows][kBtStride]
  const int b = blockIdx.z, p0 = blockIdx.x * kBtPages, tid = threadIdx.x;
  const int g = blockIdx.y % a.G, r0 = (blockIdx.y / a.G) * kBtRows;
  const int lane = tid & 31, warp = tid >> 5;
  constexpr int NW = kBtThreads / 32;
  pdl_wait();
  pdl_trigger();
  const int n_b = bs_blocks(a, b);
  if (p0 >= n_b) return;
  const int rows = min(kBtRows, a.T * a.kv_div - r0);
  // Warp w stages the blocks and the rows w, w + NW, ...; a lane 4 channels. All loads are
  // unconditional (blocks and rows past the end: the last one, not used).
  {
    constexpr int N = kBtPages / NW, R = kBtRows / NW;
    int page[N];
    float4 f[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      page[i] = a.page_table[(size_t)b * a.maxp + min(p0 + warp + i * NW, n_b - 1)];
#pragma unroll
    for (int i = 0; i < R; i += 2) {
#pragma unroll
      for (int j = i; j < i + 2; ++j) {
        const int r = warp + j * NW;
        *reinterpret_cast<float4*>(qs + r * kBtStride + 4 * lane) =
            bs_query_sum_f32<NH>(bs_query(a, b, g, r0 + min(r, rows - 1)) + 4 * lane, a.Hq / a.Gs);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool held = page[i] >= 0 && page[i] < a.n_phys;
      f[i] = ldg_f4_now(reinterpret_cast<const float4*>(
                            a.block_mean + ((size_t)(held ? page[i] : 0) * a.G + g) * kD) + lane);
    }
    float u[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (page[i] < 0 || page[i] >= a.n_phys) {
        if (lane == 0) flag_status(kStatusBadPage);
        f[i].x = __int_as_float(0x7fffffff);  // its score is NaN: it is never chosen
      }
      *reinterpret_cast<float4*>(ms + (warp + i * NW) * kBtStride + 4 * lane) = f[i];
      u[i] = fmaf(f[i].x, f[i].x, f[i].y * f[i].y) + fmaf(f[i].z, f[i].z, f[i].w * f[i].w);
    }
    if (r0 == 0) {  // the means' norms, once: lane 4 i .. 4 i + 3 end with block i's
#pragma unroll
      for (int o = 16, w = N / 2; w >= 1; o >>= 1, w >>= 1) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int k = 0; k < w; ++k) {
          const float send = upper ? u[k] : u[k + w], keep = upper ? u[k + w] : u[k];
          u[k] = keep + __shfl_xor_sync(kFull, send, o);
        }
      }
      u[0] += __shfl_xor_sync(kFull, u[0], 2);
      u[0] += __shfl_xor_sync(kFull, u[0], 1);
      const int p = p0 + warp + (lane >> 2) * NW;
      if ((lane & 3) == 0 && p < n_b) a.norms[((size_t)b * a.G + g) * a.maxp + p] = u[0];
    }
    static_assert(N == 8 && R % 2 == 0, "8 blocks per warp");
  }
  __syncthreads();
  // Threads 16 x 8: blocks tx + 16 i, rows ty + 8 j.
  const int tx = tid & 15, ty = tid >> 4;
  float acc[4][2];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[j][i] = 0.f;
#pragma unroll 1
  for (int c0 = 0; c0 < kD; c0 += 16) {
    float part[4][2];
#pragma unroll
    for (int c = c0; c < c0 + 16; c += 4) {
      float4 m[2], q[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) m[i] = *reinterpret_cast<const float4*>(ms + (tx + 16 * i) * kBtStride + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = *reinterpret_cast<const float4*>(qs + (ty + 8 * j) * kBtStride + c);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = c == c0 ? q[j].x * m[i].x : fmaf(q[j].x, m[i].x, part[j][i]);
          x = fmaf(q[j].y, m[i].y, x);
          x = fmaf(q[j].z, m[i].z, x);
          part[j][i] = fmaf(q[j].w, m[i].w, x);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[j][i] += part[j][i];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (ty + 8 * j >= rows) break;
    float* out = a.scores + bs_row(a, b, g, r0 + ty + 8 * j) * a.maxp + p0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (p0 + tx + 16 * i < n_b) out[tx + 16 * i] = acc[j][i] + 0.f;
  }
}

// One CTA per row: the m largest scores of its eligible blocks, in ascending block order.
//
// A pass over 4 NT bins of equal width between the smallest and the largest fp32 score finds the
// bin that holds the cut. The blocks within 2E of that bin's values are collected (2 to 8, for
// scores that spread); those above are kept, and unless all that were collected are kept too they
// are scored in 64 bits and ranked by (score, block). Where more than kPickMax are collected, or
// E says nothing (norms outside [1e-15, 1e18], or not finite), the whole row is scored in 64 bits
// and chosen from by block_select_largest's digit passes.
constexpr int kPickMax = 64;
// Words of dynamic shared memory: the keys, and a bit per block.
inline size_t block_topm_smem(int maxp) { return ((size_t)maxp + (maxp + 31) / 32) * 4; }
template <int NT>
__global__ void __launch_bounds__(NT) block_topm_kernel(BlockSelectArgs a) {
  __shared__ SelShared<1> sh;
  __shared__ __align__(16) int bins[4 * NT];
  __shared__ int found[4];
  __shared__ uint32_t cand_key[kPickMax];
  __shared__ int cand_at[kPickMax];
  __shared__ float nq[NT / 32], nm[NT / 32];
  extern __shared__ uint32_t bs_keys[];  // [maxp], then the bits of the taken blocks
  constexpr int NW = NT / 32, LU = 8, kBins = 4 * NT;
  uint32_t* bits = bs_keys + a.maxp;
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bt = row / a.Gs, r = row - bt * a.Gs, b = bt / a.T, g = r / a.kv_div, gs = a.Hq / a.Gs;
  const int n = eligible_blocks(a, b, bt - b * a.T), words = (n + 31) >> 5;
  int32_t* out = a.out + (size_t)row * a.m_max;
  float* sc = a.scores + (size_t)row * a.maxp;
  const float* nb = a.norms + ((size_t)b * a.G + g) * a.maxp;
  const int t = bt - b * a.T;
  const uint16_t* qrow = bs_query(a, b, g, t * a.kv_div + (r - g * a.kv_div));
  reinterpret_cast<int4*>(bins)[tid] = make_int4(0, 0, 0, 0);
  if (tid < 4) found[tid] = 0;
  float asq = 0.f;  // of ||A||
  if (tid < kD) {
#pragma unroll
    for (int h = 0; h < kMaxGroup; ++h)
      asq += h < gs ? fabsf(bf16_to_f(qrow[(size_t)h * kD + tid])) : 0.f;
    asq *= asq;
  }
  asq = warp_sum(asq);
  pdl_wait();
  pdl_trigger();

  // Keys (0: not kept whatever happens; all ones: forced) and the range of the scores.
  int live_n = 0;
  uint32_t kmin = 0xffffffffu, kmax = 0u;
  float nmax = 0.f;
  for (int base = 0; base < n; base += LU * NT) {
    float f[LU], u[LU];
#pragma unroll
    for (int j = 0; j < LU; ++j) {
      const int i = base + j * NT + tid;
      f[j] = i < n ? __ldcg(sc + i) : -INFINITY;
      u[j] = i < n ? __ldcg(nb + i) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < LU; ++j) {
      const int i = base + j * NT + tid;
      if (i >= n) break;
      const bool forced = i < a.sink || i >= n - a.local;
      const bool live = forced || f[j] > -INFINITY;
      const uint32_t kk = forced ? 0xffffffffu : live ? f2key(f[j]) : 0u;
      bs_keys[i] = kk;
      live_n += live;
      if (live && !forced) { kmin = min(kmin, kk); kmax = max(kmax, kk); }
      nmax = u[j] <= nmax ? nmax : u[j] < INFINITY ? u[j] : INFINITY;  // a NaN becomes infinite
    }
  }
  nmax = warp_max(nmax);
  if (lane == 0) {
    nq[warp] = asq;
    nm[warp] = nmax;
  }
  block_count_minmax<false>(live_n, kmin, kmax, sh.mm, &live_n, &kmin, &kmax);
  asq = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    asq += nq[w];
    nmax = fmaxf(nmax, nm[w]);
  }
  int k = min(a.m_pages, live_n);  // forced ones are at most m_pages, and all live
  const bool sound = asq > 1e-30f && asq < 1e36f && nmax > 1e-30f && nmax < 1e36f;
  auto value = [](uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
  };
  bool done = n == 0;
  // Nothing but the forced blocks is kept.
  const bool none_free = min(n, a.sink + a.local) == min(n, a.m_pages);
  if (!done && (none_free || (sound && k == live_n))) {
    for (int w = warp; w < words; w += NW) {
      const int i = 32 * w + lane;
      const uint32_t kk = i < n ? bs_keys[i] : 0u;
      const unsigned m = __ballot_sync(kFull, none_free ? kk == 0xffffffffu : kk != 0u);
      if (lane == 0) bits[w] = m;
    }
    __syncthreads();
    done = true;
  } else if (!done && sound && kmin < kmax) {
    const float lo = value(kmin), width = (value(kmax) - lo) / (kBins - 2), per = 1.f / width;
    // Not decreasing in the score; forced blocks have the last bin to themselves.
    auto bin_of = [&](uint32_t kk) {
      return kk == 0xffffffffu ? kBins - 1 : min((int)((value(kk) - lo) * per), kBins - 2);
    };
    for (int base = 0; base < n; base += LU * NT) {
      uint32_t kk[LU];
#pragma unroll
      for (int j = 0; j < LU; ++j) {
        const int i = base + j * NT + tid;
        kk[j] = i < n ? bs_keys[i] : 0u;
      }
#pragma unroll
      for (int j = 0; j < LU; ++j)
        if (kk[j] != 0u) atomicAdd(&bins[bin_of(kk[j])], 1);
    }
    __syncthreads();
    {
      // Thread t: bins 4 (NT - 1 - t) .. + 3, so that the scan runs from the top.
      const int4 c = reinterpret_cast<const int4*>(bins)[NT - 1 - tid];
      const int sum = c.x + c.y + c.z + c.w;
      int total;
      int run = block_excl_scan<false>(sum, sh.scratch, &total);
      if (run < k && k <= run + sum) {
        const int cs[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (run < k && k <= run + cs[j]) found[0] = 4 * (NT - 1 - tid) + 3 - j;
          run += cs[j];
        }
      }
    }
    __syncthreads();
    const int bin = found[0];
    // The cut lies below the forced blocks' bin: more than those are kept.
    // The bin's values, and an allowance for the rounding of bin_of, widened by 2E.
    const float e2 = 2.f * kBsErr * sqrtf(asq) * sqrtf(nmax) + 4e-6f * (fabsf(lo) + fabsf(value(kmax)));
    const float low = lo + bin * width - e2, hi = lo + (bin + 1) * width + e2;
    int sure = 0;
    for (int w0 = warp; w0 < words; w0 += LU * NW) {
      uint32_t kk[LU];
#pragma unroll
      for (int j = 0; j < LU; ++j) {
        const int i = 32 * (w0 + j * NW) + lane;
        kk[j] = i < n ? bs_keys[i] : 0u;
      }
      unsigned band_of = 0u;  // bit j: this lane's j-th block is collected
      uint32_t mine = 0u;     // lane j < LU: the j-th word
#pragma unroll
      for (int j = 0; j < LU; ++j) {
        const float s = value(kk[j]);
        const bool over = kk[j] == 0xffffffffu || (kk[j] != 0u && s > hi);
        const unsigned m = __ballot_sync(kFull, over);
        if (lane == j) mine = m;
        if (kk[j] != 0u && !over && s >= low) band_of |= 1u << j;
      }
      if (lane < LU && w0 + lane * NW < words) bits[w0 + lane * NW] = mine;
      sure += __popc(mine);
      for (; band_of != 0u; band_of &= band_of - 1u) {
        const int at = atomicAdd(&found[1], 1);  // in any order: the ranks do not depend on it
        if (at < kPickMax) cand_at[at] = 32 * (w0 + (__ffs(band_of) - 1) * NW) + lane;
      }
    }
    sure = __reduce_add_sync(kFull, sure);
    if (lane == 0) atomicAdd(&found[2], sure);
    __syncthreads();
    const int band = found[1], want = k - found[2];
    if (band <= kPickMax) {
      if (band != want) {
        double q[4];
        bs_query_sum(qrow + 4 * lane, gs, q);
        for (int c = warp; c < band; c += NW) {
          const float s = bs_exact(a, b, g, cand_at[c], q, lane);
          if (lane == 0) cand_key[c] = f2key(s);
        }
        __syncthreads();
      }
      if (tid < band) {
        const int i = cand_at[tid];
        int rank = 0;
        if (band != want)
          for (int j = 0; j < band; ++j)
            rank += cand_key[j] > cand_key[tid] || (cand_key[j] == cand_key[tid] && cand_at[j] < i);
        if (rank < want) atomicOr(&bits[i >> 5], 1u << (i & 31));
      }
      __syncthreads();
      done = true;
    }
  }
  if (!done) {
    // 64-bit scores for the whole row.
    double q[4];
    bs_query_sum(qrow + 4 * lane, gs, q);
    for (int i = warp; i < n; i += NW) {
      const float s = bs_exact(a, b, g, i, q, lane);
      if (lane == 0) sc[i] = s;
    }
    __threadfence();
    __syncthreads();
    k = block_select_largest<NT, LU, 1>(sc, n, bs_keys, sh, true, a.m_pages, 0, 0, out, a.m_max,
                                        nullptr, 0, a.sink, a.local);
  } else {
    // Warp w writes the taken blocks of the w-th part of the words.
    const int part = ceil_div(words, NW), w0 = min(words, warp * part), w1 = min(words, w0 + part);
    int before = 0;
    for (int w = lane; w < w0; w += 32) before += __popc(bits[w]);
    before = __reduce_add_sync(kFull, before);
    for (int w = w0; w < w1; w += 32) {  // a word per lane
      unsigned m = w + lane < w1 ? bits[w + lane] : 0u;
      const int incl = warp_incl_scan(__popc(m), lane);
      int at = before + incl - __popc(m);
      for (; m != 0u; m &= m - 1u) out[at++] = 32 * (w + lane) + __ffs(m) - 1;
      before += __shfl_sync(kFull, incl, 31);
    }
  }
  for (int i = k + tid; i < a.m_max; i += NT) out[i] = -1;
  if (tid == 0) a.out_count[row] = k;
}

}  // namespace hhr
