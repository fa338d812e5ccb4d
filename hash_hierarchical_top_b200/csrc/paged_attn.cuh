// Attention of one query token over whole pages of the cache: every page of a sequence (dense
// decode), or the pages of a per-query list (block-sparse decode and query chunks), from a bf16
// or an 8-bit cache.
//
// Row = one (sequence, query token, selection row): gs query heads that share the K/V rows of
// one KV head. o_h = sum_j w_hj v_j / sum_j w_hj with w_hj = exp(scale q_h . k_j - max), in one
// pass: every warp keeps a running maximum, sum and output per head (fp32) over its own keys and
// rescales them when the maximum grows; the warps of a CTA are joined in shared memory, the CTAs
// of a row by page_join_kernel.
//
// What bounds it: the K/V bytes (512 B per key and KV head in bf16, 258 B in 8 bits) against 4
// flops per byte and head, far below the tensor cores' balance. So the design keeps copies in
// flight and spends few instructions per byte:
//   - every warp runs on its own: it copies its next 16 (8-bit: 32) keys' K and V rows (8 KB) into
//     its own ring in shared memory with cp.async while it computes on the present ones; no
//     barrier in the loop, 12 warps and 96 KB in flight per SM. Loading the operands straight into
//     registers (16 warps, 128 KB) reached 5.1 TB/s where this reaches 6.8 (8 x 128K keys): it
//     spent more instructions, and its 64-byte requests split DRAM bursts.
//   - S^T = K Q^T has the keys on M = 16 and the heads on N = 8 (S = Q K^T would leave half of M
//     empty); its weights become the B operand of O^T = V^T P^T (channels on M, heads on N) by
//     one 8 x 8 transposition per 8 keys. With up to 4 heads the two parts of a weight fill the 8
//     columns of one product. Together that is half the matrix instructions of the plain layout:
//     under the 1000 W power cap the ragged 8-bit batch went from 447 to 403 us by this alone.
//   - a page id is loaded a step before the row index that needs it, and nothing loaded is looked
//     at in the step that loads it.
// P is used in parts (bf16: three, f16: two), so that the fp32 output is not limited by the matrix
// operands' type: 2e-7 to 5e-7 off the 64-bit result at 517 to 128K keys.
//
// Measured (B200, calls in a row): 8 x 128K keys x 8 KV heads in bf16 633-640 us, 6.7 TB/s of K and V
// (the measured copy rate is 6.55); 16 ragged sequences of 8K to 128K keys in 8 bits 407-414 us, 6.1
// TB/s; 1 x 32K keys 30.6 us, of which the stream takes 21; 1 x 517 keys 5.7 us, where the page table
// is no wider than 4096 keys.
//
// 8-bit cache: e4m3 numbers become f16 exactly. Q is scaled by a power of two per head so that
// its largest channel is in [2^14, 2^15): a bf16 query is then exact in f16 where its channels lie
// within 31 binades. The key's exponent multiplies its logit; the value's exponent goes into the
// weight, relative to the warp's running largest one (E_run), and 2^14 more keeps small weights
// out of f16's subnormal range: with value exponents within kPaSpread of one another, a weight is
// off by 2^-22 of itself or 2^-25 of the largest one. A warp that meets anything else (value
// exponents further apart, keys or queries that would leave fp32 on the way to an ordinary logit) has
// its keys, and in even shares its CTA's, taken again in plain fp32 (warp_fp32). 4 x 64K keys 93 us,
// with one such row in every page 651 us, with one row of zeros in every page, which only has to be
// looked at, 134 us.
//
// Split of the work: the rows' keys, in units of kUnitKeys, are laid end to end and divided
// evenly over the CTAs (three per SM), whatever the lengths; a CTA's share covers the end of one
// row, whole rows, the beginning of another. Whole rows are written directly; a share that
// covers part of a row writes a partial (at most two per CTA), joined by page_join_kernel. Short
// rows are split over a cluster instead (page_cluster_kernel).
#pragma once
#include "attn.cuh"
#include "common.cuh"
#include "kv8.cuh"

namespace hhr {

constexpr int kPaStages = 2;
constexpr int kPaWarps = 4;
constexpr int kPaThreads = kPaWarps * 32;
constexpr int kPaCtasPerSm = 3;
constexpr int kUnitKeys = 128;

struct PageAttnArgs {
  const uint16_t* q;      // [B][T][Hq][d]
  const uint16_t* k_new;  // dense: newest rows [B][G][d], appended before they are read; or null
  const uint16_t* v_new;
  void* k;                // [n_phys][G][P][d] bf16 or e4m3
  void* v;
  uint8_t* k_exp;         // 8-bit cache: [n_phys][G][P]
  uint8_t* v_exp;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* q_pos;        // [B][T] or null
  const int32_t* blocks;       // list: [B][T][Gs][m_max]
  const int32_t* block_count;  // list: [B][T][Gs]
  float* part_o;               // [2 CTAs][gs][d]
  float* part_ml;              // [2 CTAs][gs][2]
  void* out;                   // [B][T][Hq][d] f32 or bf16
  float* lse;                  // [B][T][Hq] or null
  float scale_log2;
  int out_bf16;
  int B, T, Hq, G, Gs, kv_div, P, maxp, n_phys, m_max;
  uint32_t p_mul;              // ceil(2^32 / P): j / P = umulhi(j, p_mul) for P > 1
  int n_ctas;
  uint32_t n_rows;             // n_phys G P
};

// j / P for 0 <= j < 2^24, P <= 256: p_mul exceeds 2^32 / P by less than 1, so that j p_mul / 2^32 is
// too large by less than j / 2^32 < 2^-8 <= 1 / P.
__device__ __forceinline__ int page_of(const PageAttnArgs& a, int j) {
  return a.P == 1 ? j : (int)__umulhi((uint32_t)j, a.p_mul);
}

// Keys of a dense row, and units of a row (at least one, so that an empty row is written).
__device__ __forceinline__ int dense_len(const PageAttnArgs& a, int b) {
  return min(max(a.seq_len[b], 0), a.maxp * a.P);
}
__device__ __forceinline__ int units_of(int keys) {
  return max(1, (keys + kUnitKeys - 1) / kUnitKeys);
}

// CTAs that share `total` units. Short shares (below 32 units) are a whole number per row, so that
// rows of one length are not straddled: a CTA that ends one row and begins the next fills its
// rings and joins its warps twice (2 sequences of 16K 8-bit keys: 23.4 -> 21.6 us; above, the
// CTAs left out cost more). Shares of at most two units are as few as that allows: the longest
// is no longer, and fewer partials are joined (1 sequence of 8K keys: 15.6 -> 14.6 us).
constexpr int kAlignUnits = 32;
__device__ __forceinline__ int share_count(const PageAttnArgs& a, int total) {
  const int n = min(a.n_ctas, total), rows = a.B * a.T * a.Gs;
  if (rows > n || total >= kAlignUnits * n) return n;
  const int most = n - n % rows, per = ceil_div(total, n);
  return per > 2 ? most : min(ceil_div(ceil_div(total, per), rows) * rows, most);
}
// Units of sequence b, over its rows, and the place that `pick` asks for (UnitPlace).
template <typename Pick>
__device__ __forceinline__ UnitPlace dense_place(const PageAttnArgs& a, int* sh, Pick pick) {
  return place_units(a.B, sh, [&](int b) { return units_of(dense_len(a, b)) * a.Gs; }, pick);
}

// 16 bytes into shared memory.
__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
// A word whose load is issued where it stands.
__device__ __forceinline__ uint32_t ldg_u32_now(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u32 %0, [%1];\n" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void prefetch_l1(const void* p) {
  asm volatile("prefetch.global.L1 [%0];\n" ::"l"(p) : "memory");
}
// 4 bytes into shared memory, of which the first n are read and the others are zeros.
__device__ __forceinline__ void cp_async4_zfill(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(at) : "memory");
  return v;
}
// 16 bytes into shared memory; n = 0 writes zeros and reads nothing.
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

// f16 counterpart of mma_16816, and the f16 packing of two floats.
__device__ __forceinline__ void mma_16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 2^x to 2^-22 relative; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// An 8 x 8 tile of 16-bit numbers transposed: from row lane / 4, columns 2 (lane % 4) + {0, 1}.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}
// Two weights as parts of the matrix operands' type: f16 hi + lo leave 2^-22 of a weight; bf16
// takes a third part to leave 2^-27 (two leave 2^-18, which alone put the output 1.5e-6 off).
template <bool K8>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo, uint32_t& lo2) {
  if constexpr (K8) {
    hi = pack_f16(x, y);
    const float2 h = f16x2_to_f2(hi);
    lo = pack_f16(x - h.x, y - h.y);
    lo2 = 0u;
  } else {
    hi = pack_bf16(x, y);
    const float rx = x - bf16_lo(hi), ry = y - bf16_hi(hi);  // exact
    lo = pack_bf16(rx, ry);
    lo2 = pack_bf16(rx - bf16_lo(lo), ry - bf16_hi(lo));
  }
}

// Where the keys of one row lie.
struct RowKeys {
  const int32_t* pages;   // the sequence's page-table row
  const int32_t* blocks;  // list: the row's blocks
  int n;                  // key slots: dense, the length; list, listed blocks * P
  int limit;              // keys at positions >= limit are not attended to
  uint32_t g;             // KV head
};

// Locating a key takes three steps, each of which uses what the one before it loaded. The loop
// runs them one iteration apart and leaves a loaded value alone until the next iteration (a use
// at once would stall the warp for the load's latency in every step).
// The block of slot j: dense, its page; list, the entry as it is listed (j >= k1: none).
template <bool kList>
__device__ __forceinline__ int load_block(const PageAttnArgs& a, const RowKeys& r, int j, int k1) {
  if (j >= k1) return -1;
  return kList ? r.blocks[page_of(a, j)] : page_of(a, j);
}
// The page-table entry of a loaded block; the block becomes -1 where slot j holds no key.
template <bool kList>
__device__ __forceinline__ int load_page(const PageAttnArgs& a, const RowKeys& r, int& block, int j,
                                         int k1) {
  if (kList && j < k1 && (block < 0 || block >= a.maxp)) {
    flag_status(kStatusBadToken);
    block = -1;
  }
  if (block >= 0 && block * a.P >= r.limit) block = -1;
  return block >= 0 ? r.pages[block] : 0;
}
// The cache row of slot j, or kNoRow.
__device__ __forceinline__ uint32_t row_of(const PageAttnArgs& a, const RowKeys& r, int j,
                                           int block, int page) {
  if (block < 0) return kNoRow;
  if (page < 0 || page >= a.n_phys) {
    flag_status(kStatusBadPage);
    return kNoRow;
  }
  const int slot = j - page_of(a, j) * a.P;
  if (block * a.P + slot >= r.limit) return kNoRow;
  return ((uint32_t)page * (uint32_t)a.G + r.g) * (uint32_t)a.P + (uint32_t)slot;
}

// Two query channels under a scale of 0, which leaves nothing of finite ones (their products with
// the keys might pass fp32's range); infinities and NaNs stay.
__device__ __forceinline__ uint32_t without_finite(uint32_t w) {
  return w & __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u);
}

// Shared memory of one warp: NS stages of a K tile and a V tile, S rows each (16 bf16 or
// 32 8-bit rows: 4 KB a tile). The 16-byte chunks of a row are XOR-swizzled by row % 8, so that
// ldmatrix reads of 8 rows hit 8 distinct bank groups.
// Beside the tiles lie, for an 8-bit cache, the aligned words that hold the rows' exponent bytes
// (32 of K, 32 of V): fetched like the rows, since their DRAM latency under load is longer than a
// step.
constexpr int kPaTile = 4096;
constexpr int kPaStage = 2 * kPaTile + 256;

// Row `row` (over all sequences and tokens), sequence b: where its keys are.
template <bool kList>
__device__ __forceinline__ RowKeys row_keys(const PageAttnArgs& a, int row, int b) {
  const int bt = row / a.Gs, r = row - bt * a.Gs;
  RowKeys rk;
  rk.pages = a.page_table + (size_t)b * a.maxp;
  rk.g = (uint32_t)(a.kv_div == 1 ? r : r / a.kv_div);
  rk.limit = dense_len(a, b);
  if (kList && a.q_pos != nullptr) rk.limit = min(rk.limit - 1, a.q_pos[bt]) + 1;
  rk.blocks = kList ? a.blocks + (size_t)row * a.m_max : nullptr;
  rk.n = kList ? min(max(a.block_count[row], 0), a.m_max) * a.P : rk.limit;
  if (!kList && threadIdx.x == 0 && a.seq_len[b] > a.maxp * a.P) flag_status(kStatusBadToken);
  return rk;
}

// Binades that the value exponents of one warp's keys may span in f16 weights.
constexpr uint32_t kPaSpread = 14;
// Largest exponent byte of a key whose f16 products stay in fp32: 128 of at most 2^15 448 2^96.
constexpr uint32_t kPaKeyTop = 127 + 96;
// Whether f16 holds the queries of a head whose largest |channel| has the bf16 bits `top` and whose
// smallest one that is not 0 has `low`: a head's logits are hs times products of channels times
// 2^(141 - E), E the largest one's exponent field (141 for a head of zeros). Channels may be 31
// binades apart (8 bits of each, down to 2^-24), and hs has to be a normal fp32 number.
__device__ __forceinline__ uint32_t top_exponent(uint32_t top) {
  return top == 0u ? 141u : max(top >> 7, 15u);
}
__device__ __forceinline__ float head_scale(const PageAttnArgs& a, uint32_t E) {
  return fabsf(a.scale_log2) * __uint_as_float((E - 14u) << 23);
}
__device__ __forceinline__ bool queries_far(uint32_t top, uint32_t low, float hs) {
  return top != 0u && ((top < 0x7f80u && (top >> 7) > (low >> 7) + 31u) ||
                       !(hs >= 1.17549435e-38f && hs < INFINITY));
}

// The exact way for keys and queries that f16 operands do not hold: plain fp32, on the warp's keys
// k0 .. k0 + 31, then those `step` on, below k1. Rare, so that it is no part of the kernels' loops.

// The cache row of slot j.
template <bool kList>
__device__ __forceinline__ uint32_t row_at(const PageAttnArgs& a, const RowKeys& rk, int j, int k1) {
  int block = load_block<kList>(a, rk, j, k1);
  const int page = load_page<kList>(a, rk, block, j, k1);
  return row_of(a, rk, j, block, page);
}

// Whether f16 does not hold the warp's keys under the queries q[gs][d]. page_segment asks where it has
// seen exponents far apart; it does not tell a row of zeros, which has the smallest exponent byte and
// adds nothing under any scale, from values that small.
template <bool kList>
__device__ __forceinline__ bool warp_far(const PageAttnArgs& a, const RowKeys& rk, const uint16_t* q,
                                         int gs, int k0, int step, int k1) {
  const int lane = threadIdx.x & 31;
  bool far = false;
  for (int h = 0; h < gs; ++h) {
    const uint2 w = *reinterpret_cast<const uint2*>(q + (size_t)h * kD + 4 * lane);
    uint32_t top = 0u, low = 0xffffu;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = ((i < 2 ? w.x : w.y) >> (16 * (i & 1))) & 0x7fffu;
      top = max(top, x);
      low = min(low, x - 1u);  // (0: out of the way)
    }
    top = __reduce_max_sync(kFull, top);
    low = __reduce_min_sync(kFull, low);
    far |= queries_far(top, low + 1u, head_scale(a, top_exponent(top)));
  }
  uint32_t low = 255u, high = 0u, key = 0u;
#pragma unroll 1
  for (int s0 = k0; s0 < k1; s0 += step) {
    const uint32_t row = row_at<kList>(a, rk, s0 + lane, k1);
    if (row == kNoRow) continue;
    const uint32_t x = a.v_exp[row];
    uint32_t any = 0u;
    if (x <= kExpMin) {
      const uint4* v = reinterpret_cast<const uint4*>(a.v) + (size_t)row * (kD / 16);
      for (int c = 0; c < kD / 16; ++c) any |= v[c].x | v[c].y | v[c].z | v[c].w;
    }
    if (x > kExpMin || (any & 0x7f7f7f7fu) != 0u) low = min(low, x);
    high = max(high, x);
    key = max(key, (uint32_t)a.k_exp[row]);
  }
  low = __reduce_min_sync(kFull, low);
  high = __reduce_max_sync(kFull, high);
  return far || high > low + kPaSpread || __reduce_max_sync(kFull, key) > kPaKeyTop;
}

// Attention of up to NH heads q[n][d] over the warp's keys: a lane has the channels 4 lane + {0..3} of
// o; maximum m (log2 units) and sum l of the weights. 8 keys are summed before they join the sums.
template <bool kList, int NH>
__device__ __forceinline__ void warp_fp32(const PageAttnArgs& a, const RowKeys& rk, const uint16_t* q,
                                          int n, int k0, int step, int k1, float4 (&o)[NH],
                                          float (&m)[NH], float (&l)[NH]) {
  constexpr int N = 8;
  const int lane = threadIdx.x & 31;
  float4 qf[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    uint2 w = *reinterpret_cast<const uint2*>(q + (size_t)min(h, n - 1) * kD + 4 * lane);
    if (a.scale_log2 == 0.f) w = make_uint2(without_finite(w.x), without_finite(w.y));
    qf[h] = bf16x4_to_f4(w);
    o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    m[h] = -INFINITY;
    l[h] = 0.f;
  }
  // Four e4m3 channels times 2^(x - 127).
  auto channels = [](uint32_t w, float s) {
    uint32_t lo, hi;
    e4m3x4_to_f16x2(w, lo, hi);
    const float2 x = f16x2_to_f2(lo), y = f16x2_to_f2(hi);
    return make_float4(x.x * s, x.y * s, y.x * s, y.y * s);
  };
#pragma unroll 1
  for (int s0 = k0; s0 < k1; s0 += step) {
    const uint32_t row = row_at<kList>(a, rk, s0 + lane, k1);
    const unsigned held = __ballot_sync(kFull, row != kNoRow);
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += N) {
      if ((held >> r0 & ((1u << N) - 1u)) == 0u) continue;
      uint32_t kw[N], vw[N];
      float ks[N], vs[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t r = __shfl_sync(kFull, row, r0 + i);
        const bool ok = r != kNoRow;
        const size_t at = ok ? r : 0;
        kw[i] = ok ? reinterpret_cast<const uint32_t*>(a.k)[at * (kD / 4) + lane] : 0u;
        vw[i] = ok ? reinterpret_cast<const uint32_t*>(a.v)[at * (kD / 4) + lane] : 0u;
        ks[i] = ok ? exp_scale(a.k_exp[at]) : 0.f;
        vs[i] = ok ? exp_scale(a.v_exp[at]) : 0.f;
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        if (h >= n) break;
        float x[N], top = m[h];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float4 k = channels(kw[i], ks[i]);
          x[i] = fmaf(qf[h].x, k.x, fmaf(qf[h].y, k.y, fmaf(qf[h].z, k.z, qf[h].w * k.w)));
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          x[i] = warp_sum(x[i]) * a.scale_log2;
          if (!(held >> (r0 + i) & 1u)) x[i] = -INFINITY;
          top = fmaxf(top, x[i]);
        }
        const float mu = top == -INFINITY ? 0.f : top, corr = ex2(m[h] - mu);
        m[h] = top;
        float sum = 0.f;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float w = ex2(x[i] - mu);
          const float4 v = channels(vw[i], vs[i]);
          sum += w;
          t.x = fmaf(w, v.x, t.x);
          t.y = fmaf(w, v.y, t.y);
          t.z = fmaf(w, v.z, t.z);
          t.w = fmaf(w, v.w, t.w);
        }
        l[h] = fmaf(l[h], corr, sum);
        o[h].x = fmaf(o[h].x, corr, t.x);
        o[h].y = fmaf(o[h].y, corr, t.y);
        o[h].z = fmaf(o[h].z, corr, t.z);
        o[h].w = fmaf(o[h].w, corr, t.w);
      }
    }
  }
}

// The same of a warp's part of keys [k0, k1) of a row, as page_segment deals them out.
template <bool kList>
__device__ __forceinline__ bool segment_far(const PageAttnArgs& a, int row, int b, int k0, int k1) {
  const int gs = a.Hq / a.Gs;
  const RowKeys rk = row_keys<kList>(a, row, b);
  return warp_far<kList>(a, rk, a.q + (size_t)row * gs * kD, gs, k0 + (threadIdx.x & ~31u),
                         kPaThreads, min(k1, rk.n));
}
template <bool kList>
__device__ __forceinline__ void segment_fp32(const PageAttnArgs& a, int row, int b, int k0, int k1,
                                             float* mo, float* ml) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gs = a.Hq / a.Gs;
  const RowKeys rk = row_keys<kList>(a, row, b);
  constexpr int NH = 4;
  mo += (size_t)warp * kMaxGroup * kD + 4 * lane;
  ml += warp * kMaxGroup * 2;
#pragma unroll 1
  for (int h0 = 0; h0 < gs; h0 += NH) {
    float4 o[NH];
    float m[NH], l[NH];
    warp_fp32<kList, NH>(a, rk, a.q + ((size_t)row * gs + h0) * kD, gs - h0, k0 + 32 * warp,
                         kPaThreads, min(k1, rk.n), o, m, l);
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      if (h0 + h >= gs) break;
      *reinterpret_cast<float4*>(mo + (h0 + h) * kD) = o[h];
      if (lane == 0) {
        ml[2 * (h0 + h)] = m[h];
        ml[2 * (h0 + h) + 1] = l[h];
      }
    }
  }
}
// Keys [k0, k1) of a row, over the CTA's warps: the state of every head is left in shared
// memory (mo [warps][8][d], ml [warps][8][2], which reuse the rings). True where the warp's exponents may
// be too far apart for its sums to hold (warp_far tells, warp_fp32 mends). A barrier has to follow.
// kSoon issues the query loads before the first keys are located instead of after their copies:
// a cluster's few steps gain the latency (517 keys 5.87 -> 5.72 us, lists of 64 blocks 12.85 ->
// 12.63); the shares of bf16 rows lose 1% to the registers it holds, so that they load late.
template <bool K8, bool kList, bool kPair, int NS, bool kSoon>
__device__ __forceinline__ bool page_segment(const PageAttnArgs& a, const RowKeys& rk,
                                             const uint16_t* q, int gs, int k0, int k1,
                                             char* smem, float* mo, float* ml) {
  constexpr int S = K8 ? 32 : 16;       // keys of a warp's step
  constexpr int NM = S / 16;            // 16-key tiles of S^T
  constexpr int RB = K8 ? kD : 2 * kD;  // bytes of a cache row
  constexpr int RC = RB / 16;           // 16-byte chunks of a row
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const char* kb = reinterpret_cast<const char*>(a.k);
  const char* vb = reinterpret_cast<const char*>(a.v);
  const uint32_t ring = smem_u32(smem) + (uint32_t)warp * (NS * kPaStage);
  const int base = k0 + warp * S, stride = kPaWarps * S;
  const int lk = K8 ? lane : (lane & 15);  // the key of a step that this lane locates

  // The query words of column gq (see below).
  const int head = kPair ? gq & 3 : gq;
  const bool hv = head < gs;
  uint32_t qa[8][2];
  auto load_q = [&] {
    const uint32_t* q2 = reinterpret_cast<const uint32_t*>(q + (size_t)(hv ? head : 0) * kD);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      qa[i][0] = ldg_u32_now(q2 + 8 * i + (K8 ? 2 * tq : tq));
      qa[i][1] = ldg_u32_now(q2 + 8 * i + (K8 ? 2 * tq + 1 : tq + 4));
    }
  };
  if constexpr (kSoon) load_q();

  // Copies the rows of a step (`row`: this lane's) into stage st; missing rows become zeros.
  const char* kl = kb + 16 * (lane % RC);
  const char* vl = vb + 16 * (lane % RC);
  auto issue = [&](uint32_t row, int st) {
    const uint32_t ks = ring + (uint32_t)st * kPaStage;
    if constexpr (K8) {
      const uint32_t word = row & ~3u, n = row != kNoRow ? min(4u, a.n_rows - word) : 0u;
      const uint32_t dst = ks + 2 * kPaTile + 4 * lane;
      cp_async4_zfill(dst, a.k_exp + (n != 0u ? word : 0u), n);
      cp_async4_zfill(dst + 128, a.v_exp + (n != 0u ? word : 0u), n);
    }
    if (__all_sync(kFull, row != kNoRow)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = i * (32 / RC) + lane / RC, c = lane % RC;
        const uint32_t o = __shfl_sync(kFull, row, r);
        const uint32_t dst = ks + (uint32_t)(r * RB + ((c ^ (r & 7)) << 4));
        cp_async16_at(dst, kl + (size_t)o * RB);
        cp_async16_at(dst + kPaTile, vl + (size_t)o * RB);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const int r = i * (32 / RC) + lane / RC, c = lane % RC;
        const uint32_t o = __shfl_sync(kFull, row, r);
        const uint32_t dst = ks + (uint32_t)(r * RB + ((c ^ (r & 7)) << 4));
        const uint32_t n = o != kNoRow ? 16u : 0u;
        const size_t off = o != kNoRow ? (size_t)o * RB : 0;
        cp_async16_zfill(dst, kl + off, n);
        cp_async16_zfill(dst + kPaTile, vl + off, n);
      }
    }
  };

  // rq[i]: the row this lane locates in step i from now.
  uint32_t rq[NS];
  int j0 = base + lk, blk1, page1, blk2;
  {
    int bl[NS + 1], pg[NS];
#pragma unroll
    for (int i = 0; i <= NS; ++i) bl[i] = load_block<kList>(a, rk, j0 + i * stride, k1);
#pragma unroll
    for (int i = 0; i < NS; ++i) pg[i] = load_page<kList>(a, rk, bl[i], j0 + i * stride, k1);
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) {
      rq[i] = row_of(a, rk, j0 + i * stride, bl[i], pg[i]);
      issue(rq[i], i);
      cp_async_commit();
    }
    blk1 = bl[NS - 1];
    page1 = pg[NS - 1];
    blk2 = bl[NS];
    j0 += (NS - 1) * stride;
  }
  // Query fragments of column gq: head gq, or with kPair head gq % 4 (columns without a head are
  // zero). bf16: MMA i takes the channels 16i..16i+15 in order; 8-bit: k = 2tq, 2tq + 1, 2tq + 8,
  // 2tq + 9 are the channels 16i + 4tq + {0, 1, 2, 3}.
  // A negative scale goes into the queries' signs, so that the largest product is the largest
  // logit: logit = hs * product in log2 units, hs > 0.
  if constexpr (!kSoon) load_q();
  float hs = a.scale_log2 != 0.f ? fabsf(a.scale_log2) : 1.f;
  // 8-bit: the smallest exponent byte of this lane's values, less 1 (a missing row's 0 becomes the
  // largest), and the largest one of its keys (255: queries that f16 does not hold).
  uint32_t x_low = 0xffffffffu, x_key = 0u;
  {
    const uint32_t sign = a.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      qa[i][0] = hv ? qa[i][0] ^ sign : 0u;
      qa[i][1] = hv ? qa[i][1] ^ sign : 0u;
    }
    if (a.scale_log2 == 0.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        qa[i][0] = without_finite(qa[i][0]);
        qa[i][1] = without_finite(qa[i][1]);
      }
    }
    if constexpr (K8) {
      // Bits of the largest channel (of the column) and of the smallest that is not 0 (of the lane,
      // less 1: a 0 becomes 0xffff).
      uint32_t top2 = 0u, low2 = 0xffffffffu;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t mag = qa[i][e] & 0x7fff7fffu;
          top2 = __vmaxu2(top2, mag);
          low2 = __vminu2(low2, __vsub2(mag, 0x00010001u));
        }
      uint32_t top = max(top2 & 0xffffu, top2 >> 16);
      const uint32_t low = min(low2 & 0xffffu, low2 >> 16) + 1u;
      top = max(top, __shfl_xor_sync(kFull, top, 1));
      top = max(top, __shfl_xor_sync(kFull, top, 2));
      const uint32_t E = top_exponent(top);
      const float up = __uint_as_float((268u - E) << 23);  // 2^(14 - (E - 127))
      hs = head_scale(a, E);
      if (queries_far(top, low, hs)) x_key = 255u;
      hs = fmaxf(hs, 1.17549435e-38f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        qa[i][0] = pack_f16(bf16_lo(qa[i][0]) * up, bf16_hi(qa[i][0]) * up);
        qa[i][1] = pack_f16(bf16_lo(qa[i][1]) * up, bf16_hi(qa[i][1]) * up);
      }
    }
  }

  // Of the columns 2tq + e (m_run the same on the column's 8 lanes).
  const float hse[2] = {__shfl_sync(kFull, hs, 8 * tq), __shfl_sync(kFull, hs, 8 * tq + 4)};
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
  uint32_t e_run = 0u;  // 8-bit: largest exponent byte of a value so far
  float oacc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) oacc[i][0] = oacc[i][1] = oacc[i][2] = oacc[i][3] = 0.f;
  const int l8 = lane & 7, mj = lane >> 3;  // ldmatrix: row and matrix that this lane addresses

  int st = 0;
  for (int s0 = base; s0 < k1; s0 += stride, j0 += stride) {
    cp_async_wait<NS - 2>();
    __syncwarp();  // the stage's rows are there; the previous step's stage has been read
    // The rows of NS - 1 steps ahead, and the page ids of the step after it.
    rq[NS - 1] = row_of(a, rk, j0, blk1, page1);
    issue(rq[NS - 1], st == 0 ? NS - 1 : st - 1);
    cp_async_commit();
    blk1 = blk2;
    page1 = load_page<kList>(a, rk, blk1, j0 + stride, k1);
    blk2 = load_block<kList>(a, rk, j0 + 2 * stride, k1);
    const uint32_t ks = ring + (uint32_t)st * kPaStage, vs = ks + kPaTile;
    // 8-bit: the exponent bytes of the row that this lane located (K, V); 0 for none.
    uint32_t xk = 0u, xv = 0u;
    if constexpr (K8) {
      const uint32_t at = ks + 2 * kPaTile + 4 * lane, sh = 8u * (rq[0] & 3u);
      xk = (lds_u32(at) >> sh) & 0xffu;
      xv = (lds_u32(at + 128) >> sh) & 0xffu;
    }
    const unsigned ok = __ballot_sync(kFull, rq[0] != kNoRow);

    // S^T = K Q^T, 16 keys at a time: sacc[m][2r + e] is key 16m + 8r + gq, column 2tq + e.
    float sacc[NM][4];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      float s2[4] = {0.f, 0.f, 0.f, 0.f};  // two chains of 4: less truncation, and overlap
      sacc[m][0] = sacc[m][1] = sacc[m][2] = sacc[m][3] = 0.f;
      const int r = 16 * m + (mj & 1) * 8 + l8;
#pragma unroll
      for (int c = 0; c < RC; c += 2) {  // chunks c, c + 1 of the keys 0-7 and 8-15
        uint32_t w[4];
        ldsm_x4(ks + (uint32_t)(r * RB + (((c + (mj >> 1)) ^ l8) << 4)), w[0], w[1], w[2], w[3]);
        if constexpr (K8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x2(w[2 * i], a0, a2);
            e4m3x4_to_f16x2(w[2 * i + 1], a1, a3);
            mma_16816_f16(i ? s2 : sacc[m], a0, a1, a2, a3, qa[c + i][0], qa[c + i][1]);
          }
        } else {
          mma_16816((c & 2) ? s2 : sacc[m], w[0], w[1], w[2], w[3], qa[c / 2][0], qa[c / 2][1]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sacc[m][i] += s2[i];
    }

    // 8-bit: the lane that located a key hands out 2^k_exp and what its value's weight is scaled
    // by, as two bf16 numbers.
    uint32_t ke[NM][2];
    uint32_t e_new = e_run;
    if constexpr (K8) {
      e_new = max(e_run, __reduce_max_sync(kFull, xv));
      x_low = min(x_low, xv - 1u);
      x_key = max(x_key, xk);
      const uint32_t mine = xk << 23 | (uint32_t)max(127 + 14 + (int)xv - (int)e_new, 0) << 7;
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          ke[m][r] = __shfl_sync(kFull, mine, 16 * m + 8 * r + gq);
          const float s = __uint_as_float(ke[m][r] & 0xffff0000u);
          sacc[m][2 * r] *= s;
          sacc[m][2 * r + 1] *= s;
        }
    }
    if (ok != kFull) {
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (!(ok >> (16 * m + 8 * r + gq) & 1u)) sacc[m][2 * r] = sacc[m][2 * r + 1] = -INFINITY;
    }
    float corr[2], mu[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float mx = fmaxf(sacc[0][e], sacc[0][2 + e]);
#pragma unroll
      for (int m = 1; m < NM; ++m) mx = fmaxf(mx, fmaxf(sacc[m][e], sacc[m][2 + e]));
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      // What the column's sums so far are scaled by.
      corr[e] = mx > m_run[e] ? ex2((m_run[e] - mx) * hse[e]) : 1.f;
      m_run[e] = fmaxf(m_run[e], mx);
      l_run[e] *= corr[e];
      mu[e] = m_run[e] == -INFINITY ? 0.f : -m_run[e] * hse[e];
    }
    if constexpr (K8) {
      const float ec = exp_scale((uint32_t)max(127 + (int)e_run - (int)e_new, 0));
      corr[0] *= ec;
      corr[1] *= ec;
      e_run = e_new;
    }
    // Weights, as two parts of the operands' type, transposed into B operands: ph[i] holds the
    // keys 8i + 2tq, 8i + 2tq + 1 of column gq. kPair: columns 0-3 take the first parts, 4-7 the
    // second, in one product. pm: the third parts (bf16).
    uint32_t ph[2 * NM], pl[2 * NM], pm[2 * NM];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          p[e] = ex2(fmaf(sacc[m][2 * r + e], hse[e], mu[e]));
          l_run[e] += p[e];
          if constexpr (K8) p[e] *= __uint_as_float(ke[m][r] << 16);
        }
        uint32_t hi, lo, lo2;
        split_pair<K8>(p[0], p[1], hi, lo, lo2);
        if constexpr (!K8) pm[2 * m + r] = movmatrix(kPair && tq >= 2 ? 0u : lo2);
        if constexpr (kPair) {
          ph[2 * m + r] = movmatrix(tq < 2 ? hi : lo);
        } else {
          ph[2 * m + r] = movmatrix(hi);
          pl[2 * m + r] = movmatrix(lo);
        }
      }
    // O^T = corr O^T + V^T P^T. The step's products are summed from zero and added in fp32: the
    // matrix units truncate when they add to an accumulator, and over thousands of steps that
    // is a bias (8e-6 of the output at 128K keys; 5e-7 this way).
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float o[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t w[4];
      if constexpr (K8) {
        // Chunk i of 32 keys: register k holds, for the keys 8k + 2tq and 8k + 2tq + 1, the
        // channels 16i + 2gq and 16i + 2gq + 1 (rows gq and gq + 8 of A).
        ldsm_x4_t(vs + (uint32_t)(lane * RB + ((i ^ l8) << 4)), w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x2(__byte_perm(w[2 * h], 0u, 0x3120), a0, a1);
          e4m3x4_to_f16x2(__byte_perm(w[2 * h + 1], 0u, 0x3120), a2, a3);
          mma_16816_f16(o, a0, a1, a2, a3, ph[2 * h], ph[2 * h + 1]);
          if constexpr (!kPair) mma_16816_f16(o, a0, a1, a2, a3, pl[2 * h], pl[2 * h + 1]);
        }
      } else {
        // Chunks 2i, 2i + 1 of keys 0-7, then of keys 8-15.
        const int r = (mj >> 1) * 8 + l8;
        ldsm_x4_t(vs + (uint32_t)(r * RB + (((2 * i + (mj & 1)) ^ l8) << 4)), w[0], w[1], w[2], w[3]);
        mma_16816(o, w[0], w[1], w[2], w[3], ph[0], ph[1]);
        if constexpr (!kPair) mma_16816(o, w[0], w[1], w[2], w[3], pl[0], pl[1]);
        mma_16816(o, w[0], w[1], w[2], w[3], pm[0], pm[1]);
      }
      oacc[i][0] = fmaf(oacc[i][0], corr[0], o[0]);
      oacc[i][1] = fmaf(oacc[i][1], corr[1], o[1]);
      oacc[i][2] = fmaf(oacc[i][2], corr[0], o[2]);
      oacc[i][3] = fmaf(oacc[i][3], corr[1], o[3]);
    }
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) rq[i] = rq[i + 1];
    st = st == NS - 1 ? 0 : st + 1;
  }
  cp_async_wait<0>();
  __syncthreads();  // every warp is done with its ring: mo and ml lie over them

  float* mw = mo + (size_t)warp * kMaxGroup * kD;
  float* mlw = ml + warp * kMaxGroup * 2;
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) l_run[e] += __shfl_xor_sync(kFull, l_run[e], o);
  // oacc[i]: channel c0 (elements 0, 1) and c1 (2, 3) of the columns 2tq, 2tq + 1.
  // 8-bit: 2^-14 and the running exponent, one after the other (2^(e_run - 141) may be subnormal).
  const float os = K8 ? 6.103515625e-05f : 1.f, oe = K8 ? exp_scale(e_run) : 1.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (kPair) {  // column c + 4 is the second part of column c
#pragma unroll
      for (int j = 0; j < 4; ++j) oacc[i][j] += __shfl_xor_sync(kFull, oacc[i][j], 2);
    }
    const int c0 = K8 ? 16 * i + 2 * gq : 16 * i + gq, c1 = K8 ? c0 + 1 : c0 + 8;
    if (!kPair || tq < 2) {
      mw[(2 * tq) * kD + c0] = oacc[i][0] * os * oe;
      mw[(2 * tq + 1) * kD + c0] = oacc[i][1] * os * oe;
      mw[(2 * tq) * kD + c1] = oacc[i][2] * os * oe;
      mw[(2 * tq + 1) * kD + c1] = oacc[i][3] * os * oe;
    }
  }
  if (gq == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mlw[(2 * tq + e) * 2] = m_run[e] * hse[e];  // in log2 units
      mlw[(2 * tq + e) * 2 + 1] = l_run[e];
    }
  }
  if constexpr (!K8) return false;
  return __any_sync(kFull, e_run > min(x_low, 255u) + 1u + kPaSpread || x_low < (uint32_t)kExpMin ||
                               x_key > kPaKeyTop);
}

// Writes output channel c of query head `head` (and, for c == 0, its log of the weights' sum).
__device__ __forceinline__ void put_out(const PageAttnArgs& a, size_t head, int c, float M, float L,
                                        float O) {
  const float o = L == 0.f ? 0.f : O / L;
  if (a.out_bf16)
    reinterpret_cast<__nv_bfloat16*>(a.out)[head * kD + c] = __float2bfloat16_rn(o);
  else
    reinterpret_cast<float*>(a.out)[head * kD + c] = o;
  if (c == 0 && a.lse != nullptr)
    a.lse[head] = ((M == -INFINITY ? 0.f : M) + log2f(L)) * 0.6931471805599453f;
}

// The rings; the warps' states lie over them.
inline size_t page_attn_smem() { return (size_t)kPaWarps * kPaStages * kPaStage; }
static_assert(kMaxGroup * (kD + 2) * 4 <= kPaStages * kPaStage, "a warp's state fits its ring");

// Clusters: beside the rings lies what the ranks send one another: the ranks' shares of a rank's
// outputs (at most kMaxGroup d, rounded up per rank), then per rank and head (maximum, sum).
// Three stages at two CTAs per SM are no faster (8 sequences x 64 pages: 14.3 us either way; 48
// queries x 16 pages: 24.7 us against 18.4 us).
constexpr int kPcStages = 2, kPcCtasPerSm = 3, kPaMaxCluster = 8;
constexpr int kPcShares = kMaxGroup * kD + kPaMaxCluster;                          // floats
constexpr int kPcInbox = kPcShares + 2 * kPaMaxCluster * kMaxGroup;
inline size_t page_cluster_smem() {
  return (size_t)kPaWarps * kPcStages * kPaStage + (size_t)kPcInbox * 4;
}

// Dense: writes the newest row (position rk.n - 1) of sequence b into the cache; by the CTA that
// reads it, before the barrier behind which it does. A length past the page table has no such row.
template <bool K8>
__device__ __forceinline__ void append_row(const PageAttnArgs& a, const RowKeys& rk, int b) {
  const int tid = threadIdx.x, t = rk.n - 1, l16 = tid & 15;
  if (tid >= 32 || a.seq_len[b] > a.maxp * a.P) return;
  int lp = page_of(a, t);
  const int page = load_page<false>(a, rk, lp, t, rk.n);
  const uint32_t o = row_of(a, rk, t, lp, page);
  if (o == kNoRow) return;
  const uint16_t* src = (tid < 16 ? a.k_new : a.v_new) + ((size_t)b * a.G + rk.g) * kD;
  char* dst = reinterpret_cast<char*>(tid < 16 ? a.k : a.v);
  const uint4 w = reinterpret_cast<const uint4*>(src)[l16];
  if constexpr (K8) {
    const uint32_t x = row_exponent(row_top16(w, 0xffffu << (tid & 16)));
    *reinterpret_cast<uint2*>(dst + (size_t)o * kD + 8 * l16) = quantise8(w, x);
    if (l16 == 0) (tid < 16 ? a.k_exp : a.v_exp)[o] = (uint8_t)x;
  } else {
    *reinterpret_cast<uint4*>(dst + (size_t)o * 2 * kD + 16 * l16) = w;
  }
}

// Joins the warps' states: put(h, channel, M, L, O) for every head, thread t taking channel t.
static_assert(kPaThreads == kD, "a thread per channel");
template <typename Put>
__device__ __forceinline__ void join_warps(const float* mo, const float* ml, int gs, Put put) {
  const int ch = threadIdx.x;
#pragma unroll 4
  for (int h = 0; h < gs; ++h) {
    float m[kPaWarps], M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kPaWarps; ++w) {
      m[w] = ml[(w * kMaxGroup + h) * 2];
      M = fmaxf(M, m[w]);
    }
    const float mu = M == -INFINITY ? 0.f : M;
    float L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < kPaWarps; ++w) {
      const float f = ex2(m[w] - mu);
      L = fmaf(f, ml[(w * kMaxGroup + h) * 2 + 1], L);
      O = fmaf(f, mo[((size_t)w * kMaxGroup + h) * kD + ch], O);
    }
    put(h, ch, M, L, O);
  }
}

// A CTA's even share of all rows' keys (see the head of this file), of which units [off, off + take())
// of row `row` (over all sequences and tokens; sequence b) come next.
struct Share {
  int u, end, row, b, off, ub;  // units [u, end) are left; ub: units of the row
  __device__ __forceinline__ int take() const { return min(end - u, ub - off); }
};
// False: this CTA has no share. Block-wide; sh: 40 ints.
template <bool kList>
__device__ __forceinline__ bool share_start(const PageAttnArgs& a, int* sh, Share& s) {
  const int c = blockIdx.x;
  int total;
  if (kList) {
    s.ub = units_of(a.m_max * a.P);
    total = a.B * a.T * a.Gs * s.ub;
  } else {
    const UnitPlace p = dense_place(a, sh, [&](int all) {
      return min(share_begin(c, all, share_count(a, all)), all - 1);
    });
    total = p.total;
    s.b = p.b;
    s.off = p.before;
  }
  const int n = share_count(a, total);
  if (c >= n) return false;
  s.u = share_begin(c, total, n);
  s.end = share_begin(c + 1, total, n);
  if (kList) {
    s.row = s.u / s.ub;
    s.off = s.u - s.row * s.ub;
    s.b = s.row / a.Gs / a.T;
  } else {
    s.ub = units_of(dense_len(a, s.b));
    s.row = s.b * a.Gs + (s.u - s.off) / s.ub;
    s.off = (s.u - s.off) % s.ub;
  }
  return true;
}
// On to the next row; false at the share's end.
template <bool kList>
__device__ __forceinline__ bool share_next(const PageAttnArgs& a, Share& s) {
  s.u += s.take();
  if (s.u >= s.end) return false;
  ++s.row;
  s.off = 0;
  s.b = kList ? s.row / a.Gs / a.T : s.row / a.Gs;
  if (!kList) s.ub = units_of(dense_len(a, s.b));
  return true;
}
// Writes what the CTA's warps have of the share's part: the outputs of a whole row, else a partial.
__device__ __forceinline__ void put_part(const PageAttnArgs& a, const Share& s, const float* mo,
                                         const float* ml) {
  const int gs = a.Hq / a.Gs;
  const bool whole = s.off == 0 && s.take() == s.ub;
  const size_t slot = 2 * (size_t)blockIdx.x + (s.off == 0 ? 1 : 0);
  join_warps(mo, ml, gs, [&](int h, int ch, float M, float L, float O) {
    if (whole) {
      put_out(a, (size_t)s.row * gs + h, ch, M, L, O);
    } else {
      a.part_o[(slot * gs + h) * kD + ch] = O;
      if (ch == 0) {
        a.part_ml[(slot * gs + h) * 2] = M;
        a.part_ml[(slot * gs + h) * 2 + 1] = L;
      }
    }
  });
}

// The CTA's share once more, where f16 operands do not hold a part of it: the last thing that the
// kernel does, so that its loop keeps nothing in registers for the call (a call per part made lists
// of 64 queries 4% slower; so did arguments by reference).
template <bool kList>
__device__ __noinline__ void page_share_fp32(PageAttnArgs a, int* sh, float* mo, float* ml) {
  Share s;
  if (!share_start<kList>(a, sh, s)) return;
  do {
    const int k0 = s.off * kUnitKeys, k1 = k0 + s.take() * kUnitKeys;
    if (!__syncthreads_or(segment_far<kList>(a, s.row, s.b, k0, k1))) continue;
    segment_fp32<kList>(a, s.row, s.b, k0, k1, mo, ml);
    __syncthreads();
    put_part(a, s, mo, ml);
  } while (share_next<kList>(a, s));
}

template <bool K8, bool kList, bool kPair>
__global__ void __launch_bounds__(kPaThreads, kPaCtasPerSm) page_attn_kernel(PageAttnArgs a) {
  pdl_wait();
  extern __shared__ float4 pa_smem[];
  __shared__ int sh[40];
  float* mo = reinterpret_cast<float*>(pa_smem);
  float* ml = mo + kPaWarps * kMaxGroup * kD;
  const int gs = a.Hq / a.Gs;
  pdl_trigger();  // page_join_kernel waits for this grid's end before it reads the partials
  Share s;
  if (!share_start<kList>(a, sh, s)) return;
  bool far = false;
  do {
    const RowKeys rk = row_keys<kList>(a, s.row, s.b);
    const int take = s.take();
    if (!kList && a.k_new != nullptr && s.off + take == s.ub && rk.n > 0) append_row<K8>(a, rk, s.b);
    __syncthreads();  // the new row is visible; the previous segment's state has been read
    far |= page_segment<K8, kList, kPair, kPaStages, K8>(
        a, rk, a.q + (size_t)s.row * gs * kD, gs, s.off * kUnitKeys,
        min(rk.n, (s.off + take) * kUnitKeys), reinterpret_cast<char*>(pa_smem), mo, ml);
    __syncthreads();
    put_part(a, s, mo, ml);
  } while (share_next<kList>(a, s));
  if constexpr (K8)
    if (__syncthreads_or(far)) page_share_fp32<kList>(a, sh, mo, ml);
}

// The keys [k0, k1) of a row that rank `rank` of its cluster of cs CTAs takes: equal parts, whole
// iterations of a CTA.
template <bool K8>
__device__ __forceinline__ int2 cluster_keys(int n, int cs, int rank) {
  constexpr int kIter = kPaWarps * (K8 ? 32 : 16);
  const int per = ceil_div(ceil_div(n, cs), kIter) * kIter;
  const int k0 = min(n, rank * per);
  return make_int2(k0, min(n, k0 + per));
}
// A cluster's warp whose exponents page_segment found far apart: looks, and replaces its state. Not
// inlined, and finding its place itself, to stay out of page_segment's registers (place passed: up to
// 2000 keys of 8 sequences, 8 heads per KV head, 15.6 us; this way 14.9; without the call 14.4).
template <bool kList>
__device__ __noinline__ void page_segment_fp32(PageAttnArgs a, float* mo) {
  namespace cg = cooperative_groups;
  cg::cluster_group cl = cg::this_cluster();
  const int cs = (int)cl.num_blocks(), row = blockIdx.x / cs, b = row / a.Gs / a.T;
  const int2 keys = cluster_keys<true>(row_keys<kList>(a, row, b).n, cs, (int)cl.block_rank());
  if (!segment_far<kList>(a, row, b, keys.x, keys.y)) return;
  __syncwarp();  // the state that is replaced has been written
  segment_fp32<kList>(a, row, b, keys.x, keys.y, mo, mo + kPaWarps * kMaxGroup * kD);
}

// One cluster per row: its CTAs take equal parts of the row's keys. Rank r writes the r-th part of
// the row's outputs: every rank sends it that part of its state through distributed shared memory,
// into an inbox beside the rings. One launch, no partials in global memory.
template <bool K8, bool kList, bool kPair>
__global__ void __launch_bounds__(kPaThreads, kPcCtasPerSm) page_cluster_kernel(PageAttnArgs a) {
  pdl_wait();
  pdl_trigger();
  namespace cg = cooperative_groups;
  extern __shared__ float4 pa_smem[];
  cluster_arrive();  // waited for before the first remote write: every rank has started
  float* mo = reinterpret_cast<float*>(pa_smem);
  float* ml = mo + kPaWarps * kMaxGroup * kD;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, gs = a.Hq / a.Gs;
  const int cs = (int)cl.num_blocks(), rank = (int)cl.block_rank(), row = blockIdx.x / cs;
  const int bt = row / a.Gs, r = row - bt * a.Gs, b = bt / a.T;
  // Slot s of the inbox: rank s's share of this rank's outputs ([part]), and its (M, L) per head.
  const int part = ceil_div(gs * kD, cs);
  float* inbox = reinterpret_cast<float*>(reinterpret_cast<char*>(pa_smem) +
                                          (size_t)kPaWarps * kPcStages * kPaStage);
  float* inbox_ml = inbox + kPcShares;
  // Where the keys lie takes three dependent loads (length, block or page id, key): the page ids
  // and the block list are brought into L1 while the length is on its way.
  if (32 * tid < a.maxp) prefetch_l1(a.page_table + (size_t)b * a.maxp + 32 * tid);
  if (kList && 32 * tid < a.m_max) prefetch_l1(a.blocks + (size_t)row * a.m_max + 32 * tid);
  const RowKeys rk = row_keys<kList>(a, row, b);
  const int2 keys = cluster_keys<K8>(rk.n, cs, rank);
  const int k0 = keys.x, k1 = keys.y;
  if (!kList && a.k_new != nullptr && k0 < k1 && k1 == rk.n) append_row<K8>(a, rk, b);
  __syncthreads();
  const size_t head0 = (size_t)bt * a.Hq + (size_t)r * gs;
  if (page_segment<K8, kList, kPair, kPcStages, true>(a, rk, a.q + head0 * kD, gs, k0, k1,
                                                      reinterpret_cast<char*>(pa_smem), mo, ml))
    page_segment_fp32<kList>(a, mo);
  __syncthreads();
  cluster_wait();
  const float per_part = 1.f / (float)part;
  join_warps(mo, ml, gs, [&](int h, int ch, float M, float L, float O) {
    // i / part: i + 1/2 is no nearer to a multiple of part than 1/2, so the rounding is harmless.
    const int i = h * kD + ch, to = (int)(((float)i + 0.5f) * per_part);
    *cl.map_shared_rank(inbox + rank * part + (i - to * part), to) = O;
    if (ch < cs) {  // (M, L) of the head, once to each rank
      float* x = cl.map_shared_rank(inbox_ml + (rank * kMaxGroup + h) * 2, ch);
      x[0] = M;
      x[1] = L;
    }
  });
  cluster_sync_all();  // every rank's share has arrived; no remote access follows
  const int n = min(part, gs * kD - rank * part);
  for (int j = tid; j < n; j += kPaThreads) {
    const int i = rank * part + j, h = i / kD;
    float m[kPaMaxCluster], M = -INFINITY;
#pragma unroll
    for (int c = 0; c < kPaMaxCluster; ++c) {
      m[c] = c < cs ? inbox_ml[(c * kMaxGroup + h) * 2] : -INFINITY;
      M = fmaxf(M, m[c]);
    }
    const float mu = M == -INFINITY ? 0.f : M;
    float L = 0.f, O = 0.f;
#pragma unroll
    for (int c = 0; c < kPaMaxCluster; ++c) {
      if (c < cs) {
        const float f = ex2(m[c] - mu);
        L = fmaf(f, inbox_ml[(c * kMaxGroup + h) * 2 + 1], L);
        O = fmaf(f, inbox[c * part + j], O);
      }
    }
    put_out(a, head0 + h, i % kD, M, L, O);
  }
}

// Joins the partials of one row and head: the CTAs c0..c1 whose shares touch the row, the first
// of them with its "row begins here" slot, the others with their "row goes on" slot. Grid (row,
// head of the row); rows that one CTA covered are already written. The weights 2^(m - M) are
// taken once per partial, by one thread each; then warp w sums the partials w, w + 8, ..., a lane
// holding 4 channels, and the 8 sums are added in order.
constexpr int kJoinWarps = 8;
constexpr int kJoinThreads = kJoinWarps * 32;
constexpr int kJoinChunk = kJoinThreads;  // partials whose weights are in shared memory at a time
template <bool kList>
__global__ void __launch_bounds__(kJoinThreads) page_join_kernel(PageAttnArgs a) {
  __shared__ int sh[40];
  __shared__ float wt[kJoinChunk], red[2][kJoinWarps];
  __shared__ __align__(16) float acc[kJoinWarps][kD];
  const int row = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, gs = a.Hq / a.Gs;
  const int lane = tid & 31, warp = tid >> 5;
  int total, first, ub;
  if (kList) {
    ub = units_of(a.m_max * a.P);
    total = a.B * a.T * a.Gs * ub;
    first = row * ub;
  } else {
    const int bs = row / a.Gs;
    const UnitPlace p = dense_place(a, sh, [&](int) { return -1 - bs; });
    total = p.total;
    ub = units_of(dense_len(a, bs));
    first = p.before + (row - bs * a.Gs) * ub;
  }
  const int n = share_count(a, total);
  const int c0 = share_of(first, total, n), parts = share_of(first + ub - 1, total, n) - c0 + 1;
  pdl_wait();
  pdl_trigger();
  if (parts == 1) return;
  auto slot = [&](int i) { return ((size_t)2 * (c0 + i) + (i == 0 ? 1 : 0)) * gs + h; };
  float M = -INFINITY;
  for (int i = tid; i < parts; i += kJoinThreads) M = fmaxf(M, __ldcg(a.part_ml + slot(i) * 2));
  M = warp_max(M);
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, red[0][w]);
  const float mu = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < parts; i0 += kJoinChunk) {
    if (i0 > 0) __syncthreads();
    if (i0 + tid < parts) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + slot(i0 + tid));
      wt[tid] = exp2f(ml.x - mu);
      L = fmaf(wt[tid], ml.y, L);
    }
    __syncthreads();
    const int k = min(kJoinChunk, parts - i0);
#pragma unroll 4
    for (int i = warp; i < k; i += kJoinWarps) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + slot(i0 + i) * kD) + lane);
      const float f = wt[i];
      o.x = fmaf(f, v.x, o.x);
      o.y = fmaf(f, v.y, o.y);
      o.z = fmaf(f, v.z, o.z);
      o.w = fmaf(f, v.w, o.w);
    }
  }
  reinterpret_cast<float4*>(acc[warp])[lane] = o;
  L = warp_sum(L);
  if (lane == 0) red[1][warp] = L;
  __syncthreads();
  if (tid < kD) {
    float O = 0.f;
    L = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      O += acc[w][tid];
      L += red[1][w];
    }
    const int bt = row / a.Gs, r = row - bt * a.Gs;
    put_out(a, (size_t)bt * a.Hq + (size_t)r * gs + h, tid, M, L, O);
  }
}

}  // namespace hhr
