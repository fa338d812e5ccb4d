// The 8-bit K/V cache: rows quantised as they are appended, and read back.
//
// A row x of 128 channels is held as 128 e4m3 numbers q and one exponent byte: x ~ q 2^e, byte
// = e + 127, with e the smallest whole number of [-117, 119] such that max|x| <= 448 2^e (448 =
// the largest e4m3 number). A power of two loses no precision against max|x| / 448: e4m3 is a
// floating-point format of 17 binades, and the scaled maximum lies in its top one. In exchange
// the division is exact, every channel is rounded once (to nearest even, half a step of 2^-4
// relative, or 2^-10 absolute in q below 2^-6), and q 2^e is a bf16 number exactly, so reading
// back loses nothing. The byte is also the exponent field of the float 2^e.
//
// Both kernels only move bytes: 256 B read and 129 B written per row, or the reverse.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace hhr {

constexpr int kExpMin = 127 - 117, kExpMax = 127 + 119;  // exponent bytes

// 2^(x - 127) of an exponent byte.
__device__ __forceinline__ float exp_scale(uint32_t x) { return __uint_as_float(x << 23); }

// Exponent byte of a row whose largest |channel| has the bf16 bits `top` (sign clear). With
// top = (1 + m/128) 2^(E - 127): 448 = 1.75 * 2^8, so e = E - 127 - 8, one more when the
// significand is above 1.75. An infinity takes the largest byte and is then saturated.
__device__ __forceinline__ uint32_t row_exponent(uint32_t top) {
  const int x = (int)(top >> 7) - 8 + ((top & 127u) > 96u ? 1 : 0);
  return (uint32_t)min(max(x, kExpMin), kExpMax);
}

// The larger of two pairs of bf16 numbers; a NaN only where both are.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Largest |channel| (bf16 bits; NaNs ignored) of the row that 16 lanes hold, 8 channels each.
__device__ __forceinline__ uint32_t row_top16(uint4 w, unsigned mask) {
  constexpr uint32_t kAbs = 0x7fff7fffu;
  uint32_t m = max_bf16x2(max_bf16x2(w.x & kAbs, w.y & kAbs), max_bf16x2(w.z & kAbs, w.w & kAbs));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_bf16x2(m, __shfl_xor_sync(mask, m, o));
  const uint32_t lo = m & 0xffffu, hi = m >> 16;  // above 0x7f80: nothing but NaNs
  return max(lo > 0x7f80u ? 0u : lo, hi > 0x7f80u ? 0u : hi);
}

// Two floats to e4m3 (to nearest even, saturating; NaN stays NaN): a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// Two e4m3 bytes (low 16 bits) to f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
// Four e4m3 bytes to two f16x2.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float2 f16x2_to_f2(uint32_t two) {
  return __half22float2(*reinterpret_cast<const __half2*>(&two));
}

// 8 bf16 channels times 2^-e, rounded to e4m3.
__device__ __forceinline__ uint2 quantise8(uint4 w, uint32_t x) {
  const float s = __uint_as_float((254u - x) << 23);  // 2^-(x - 127)
  uint2 r;
  r.x = e4m3x2(bf16_lo(w.x) * s, bf16_hi(w.x) * s) | e4m3x2(bf16_lo(w.y) * s, bf16_hi(w.y) * s) << 16;
  r.y = e4m3x2(bf16_lo(w.z) * s, bf16_hi(w.z) * s) | e4m3x2(bf16_lo(w.w) * s, bf16_hi(w.w) * s) << 16;
  return r;
}

// 16 bytes that are read once; the load is issued where it stands.
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

struct AppendArgs {
  const uint16_t* k_new;  // token i of sequence b, head g: + (b * max_new + i) * stride + g * d
  const uint16_t* v_new;
  const int32_t* start;
  const int32_t* n_new;
  const int32_t* page_table;
  uint8_t* k;  // [n_phys][G][P][d]
  uint8_t* v;
  uint8_t* k_exp;  // [n_phys][G][P]
  uint8_t* v_exp;
  float* block_mean;  // [n_phys][G][d] or null
  long long stride;
  int G, P, maxp, n_phys, max_new;
};

constexpr int kAppendThreads = 128;
constexpr int kAppendRows = kAppendThreads / 16;  // rows per pass: 16 lanes each
constexpr int kAppendUnroll = 2;

// One CTA per (touched page, KV group, sequence). 16 lanes quantise a row, 8 channels a lane.
// A prefill is bound by instructions as much as by its bytes: 178K rows of K and V take 27.7 us (137
// MB, 4.95 TB/s, 75% of the copy rate); 41 us with scalar maxima, one tensor after the other and
// CTAs of 256 threads. A token per sequence takes 3.3 us, all of it latency.
// With block_mean, the K rows that the page held before are read too, and the mean is taken
// over the values that the cache stands for.
template <bool kMean>
__global__ void __launch_bounds__(kAppendThreads) append_kv8_kernel(AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float part[kMean ? kAppendRows : 1][kD];
  const int b = blockIdx.z, g = blockIdx.y, tid = threadIdx.x;
  const int P = a.P;
  int nn = a.n_new[b];
  if (nn > a.max_new) {
    if (tid == 0 && blockIdx.x == 0 && g == 0) flag_status(kStatusClipped);
    nn = a.max_new;
  }
  const int s = a.start[b];
  if (nn <= 0 || s < 0) return;
  const long long e = (long long)s + nn;
  const long long lp = s / P + (long long)blockIdx.x;
  if (lp * P >= e) return;
  if (lp >= a.maxp) {
    if (tid == 0) flag_status(kStatusBadPage);
    return;
  }
  // Not looked at before the first rows are on their way: one latency less per CTA.
  const int phys = a.page_table[(size_t)b * a.maxp + lp];
  const int pstart = (int)lp * P;
  const int t0 = max(s, pstart) - pstart, t1 = (int)min(e, (long long)pstart + P) - pstart;
  const int lane = tid & 15, sub = tid >> 4;
  const unsigned mask = 0xffffu << (tid & 16);  // the row's 16 lanes
  size_t row0 = 0;
  const size_t src0 = ((size_t)b * a.max_new + (pstart + t0 - s)) * a.stride + (size_t)g * kD + 8 * lane;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  auto add = [&](uint2 q, uint32_t x) {
    const float sc = exp_scale(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = f16x2_to_f2(e4m3x2_to_f16x2((i < 2 ? q.x : q.y) >> (16 * (i & 1))));
      sum[2 * i] = fmaf(f.x, sc, sum[2 * i]);
      sum[2 * i + 1] = fmaf(f.y, sc, sum[2 * i + 1]);
    }
  };
  // New rows, kAppendUnroll of K and of V at a time: their loads are in flight together.
  constexpr int U = kAppendUnroll;
  for (int r0 = t0 + sub; r0 - sub < t1; r0 += U * kAppendRows) {  // the same steps for all threads
    uint4 w[2][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * kAppendRows;
      const size_t src = src0 + (size_t)(r - t0) * a.stride;
      w[0][u] = r < t1 ? ldg_stream(a.k_new + src) : make_uint4(0u, 0u, 0u, 0u);
      w[1][u] = r < t1 ? ldg_stream(a.v_new + src) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (phys < 0 || phys >= a.n_phys) {
      if (tid == 0) flag_status(kStatusBadPage);
      return;
    }
    row0 = ((size_t)phys * a.G + g) * P;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t row = row0 + r0 + u * kAppendRows;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t x = row_exponent(row_top16(w[kv][u], mask));
        const uint2 q = quantise8(w[kv][u], x);
        if (r0 + u * kAppendRows < t1) {
          *reinterpret_cast<uint2*>((kv ? a.v : a.k) + row * kD + 8 * lane) = q;
          if (lane == 0) (kv ? a.v_exp : a.k_exp)[row] = (uint8_t)x;
          if (kMean && kv == 0) add(q, x);
        }
      }
    }
  }
  if constexpr (kMean) {
    for (int r0 = sub; r0 < t0; r0 += U * kAppendRows) {  // what the page held before
      uint2 q[U];
      uint32_t x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * kAppendRows;
        q[u] = r < t0 ? *reinterpret_cast<const uint2*>(a.k + (row0 + r) * kD + 8 * lane)
                      : make_uint2(0u, 0u);
        x[u] = r < t0 ? a.k_exp[row0 + r] : 0u;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) add(q[u], x[u]);
    }
  }
  if constexpr (kMean) {
#pragma unroll
    for (int i = 0; i < 8; ++i) part[sub][8 * lane + i] = sum[i];
    __syncthreads();
    if (tid < kD) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < kAppendRows; ++i) t += part[i][tid];
      a.block_mean[((size_t)phys * a.G + g) * kD + tid] = t / (float)t1;
    }
  }
}

struct ReadArgs {
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  const int32_t* page_table;
  const int32_t* start;
  const int32_t* n;
  uint16_t* k_out;  // [B][max_n][G][d]
  uint16_t* v_out;
  int G, P, maxp, n_phys, max_n;
  uint32_t p_mul;  // ceil(2^32 / P)
};

constexpr int kReadThreads = 256;
constexpr int kReadRows = kReadThreads / 16;  // rows per pass: 16 lanes each, 8 channels a lane
constexpr int kReadUnroll = 2;  // 1: 144 us, 4: 137 us where 2 takes 136
constexpr int kReadTile = kReadRows * kReadUnroll;

// 8 e4m3 channels times 2^(x - 127), as bf16 (exact).
__device__ __forceinline__ uint4 dequantise8(uint2 q, uint32_t x) {
  const float s = exp_scale(x);
  auto two = [&](uint32_t f16) {
    const float2 f = f16x2_to_f2(f16);
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * s, f.y * s);
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  uint32_t a, b, c, d;
  e4m3x4_to_f16x2(q.x, a, b);
  e4m3x4_to_f16x2(q.y, c, d);
  return make_uint4(two(a), two(b), two(c), two(d));
}

// Grid (rows / kReadTile, KV group, sequence). A lane writes 16 bytes next to its neighbour's 16
// (with 32 a lane in two stores, every 32-byte sector was written in halves: 150 us where this
// takes 134 us, 4 sequences of 32K keys: 6.0 TB/s of the bytes read and written, 92% of the copy
// rate). Bound by those bytes.
__global__ void __launch_bounds__(kReadThreads) read_kv8_kernel(ReadArgs a) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z, g = blockIdx.y, tid = threadIdx.x;
  int n = a.n[b];
  if (n > a.max_n) {
    if (tid == 0 && blockIdx.x == 0 && g == 0) flag_status(kStatusClipped);
    n = a.max_n;
  }
  const int i0 = blockIdx.x * kReadTile + (tid >> 4), lane = tid & 15;
  if (i0 >= n) return;
  const long long start = a.start[b];
  constexpr int U = kReadUnroll;
  constexpr uint32_t kNone = 0xffffffffu;
  uint32_t row[U];  // cache row, or kNone
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = i0 + u * kReadRows;
    const long long t = start + i;
    row[u] = kNone;
    if (i >= n) continue;
    if (t < 0 || t >= a.maxp * a.P) {
      if (lane == 0) flag_status(kStatusBadToken);
      continue;
    }
    // t / P: t < 2^23 and P <= 256, so the product is too large by less than 2^-9 < 1 / P.
    const int lp = a.P == 1 ? (int)t : (int)__umulhi((uint32_t)t, a.p_mul);
    const int phys = a.page_table[(size_t)b * a.maxp + lp];
    if (phys < 0 || phys >= a.n_phys) {
      if (lane == 0) flag_status(kStatusBadPage);
      continue;
    }
    row[u] = ((uint32_t)phys * (uint32_t)a.G + g) * (uint32_t)a.P + (uint32_t)((int)t - lp * a.P);
  }
  uint2 q[2][U];
  uint32_t x[2][U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row[u] == kNone) continue;
    q[0][u] = *reinterpret_cast<const uint2*>(a.k + (size_t)row[u] * kD + 8 * lane);
    q[1][u] = *reinterpret_cast<const uint2*>(a.v + (size_t)row[u] * kD + 8 * lane);
    x[0][u] = a.k_exp[row[u]];
    x[1][u] = a.v_exp[row[u]];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row[u] == kNone) continue;
    const size_t o = (((size_t)b * a.max_n + (i0 + u * kReadRows)) * a.G + g) * kD + 8 * lane;
    *reinterpret_cast<uint4*>(a.k_out + o) = dequantise8(q[0][u], x[0][u]);
    *reinterpret_cast<uint4*>(a.v_out + o) = dequantise8(q[1][u], x[1][u]);
  }
}

}  // namespace hhr
