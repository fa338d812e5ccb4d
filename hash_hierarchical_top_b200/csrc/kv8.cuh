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

// Largest |channel| (bf16 bits; NaNs ignored) of the row that 16 lanes hold, 8 channels each.
__device__ __forceinline__ uint32_t row_top16(uint4 w, unsigned mask) {
  auto mag = [](uint32_t two) {  // |.| of both halves; a NaN counts as 0
    uint32_t lo = two & 0x7fffu, hi = (two >> 16) & 0x7fffu;
    if (lo > 0x7f80u) lo = 0u;
    if (hi > 0x7f80u) hi = 0u;
    return max(lo, hi);
  };
  uint32_t m = max(max(mag(w.x), mag(w.y)), max(mag(w.z), mag(w.w)));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
  return m;
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

constexpr int kAppendThreads = 256;
constexpr int kAppendRows = kAppendThreads / 16;  // rows in flight: 16 lanes each

// One CTA per (touched page, KV group, sequence). 16 lanes quantise a row, 8 channels a lane.
// With block_mean, the K rows that the page held before are read too, and the mean is taken
// over the values that the cache stands for.
template <bool kMean>
__global__ void __launch_bounds__(kAppendThreads) append_kv8_kernel(AppendArgs a) {
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
  const int phys = a.page_table[(size_t)b * a.maxp + lp];
  if (phys < 0 || phys >= a.n_phys) {
    if (tid == 0) flag_status(kStatusBadPage);
    return;
  }
  const int pstart = (int)lp * P;
  const int t0 = max(s, pstart) - pstart, t1 = (int)min(e, (long long)pstart + P) - pstart;
  const int lane = tid & 15, sub = tid >> 4;
  const unsigned mask = 0xffffu << (tid & 16);  // the row's 16 lanes
  const size_t row0 = ((size_t)phys * a.G + g) * P;
  const size_t src0 = ((size_t)b * a.max_new + (pstart + t0 - s)) * a.stride + (size_t)g * kD + 8 * lane;
  // V rows, then K rows.
  for (int r = t0 + sub; r < t1; r += kAppendRows) {
    const uint4 w = *reinterpret_cast<const uint4*>(a.v_new + src0 + (size_t)(r - t0) * a.stride);
    const uint32_t x = row_exponent(row_top16(w, mask));
    *reinterpret_cast<uint2*>(a.v + (row0 + r) * kD + 8 * lane) = quantise8(w, x);
    if (lane == 0) a.v_exp[row0 + r] = (uint8_t)x;
  }
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  for (int r = (kMean ? 0 : t0) + sub; r < t1; r += kAppendRows) {
    uint2 q;
    uint32_t x;
    if (kMean && r < t0) {
      q = *reinterpret_cast<const uint2*>(a.k + (row0 + r) * kD + 8 * lane);
      x = a.k_exp[row0 + r];
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(a.k_new + src0 + (size_t)(r - t0) * a.stride);
      x = row_exponent(row_top16(w, mask));
      q = quantise8(w, x);
      *reinterpret_cast<uint2*>(a.k + (row0 + r) * kD + 8 * lane) = q;
      if (lane == 0) a.k_exp[row0 + r] = (uint8_t)x;
    }
    if constexpr (kMean) {
      const float sc = exp_scale(x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = f16x2_to_f2(e4m3x2_to_f16x2((i < 2 ? q.x : q.y) >> (16 * (i & 1))));
        sum[2 * i] = fmaf(f.x, sc, sum[2 * i]);
        sum[2 * i + 1] = fmaf(f.y, sc, sum[2 * i + 1]);
      }
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
};

constexpr int kReadThreads = 256;
constexpr int kReadRows = kReadThreads / 8;  // rows per pass: 8 lanes each, 16 channels a lane

// 16 e4m3 channels times 2^(x - 127), as bf16 (exact).
__device__ __forceinline__ void dequantise16(uint4 q, uint32_t x, uint4& lo, uint4& hi) {
  const float s = exp_scale(x);
  auto two = [&](uint32_t w, int half) {
    const float2 f = f16x2_to_f2(e4m3x2_to_f16x2(w >> (16 * half)));
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * s, f.y * s);
    return *reinterpret_cast<const uint32_t*>(&r);
  };
  lo = make_uint4(two(q.x, 0), two(q.x, 1), two(q.y, 0), two(q.y, 1));
  hi = make_uint4(two(q.z, 0), two(q.z, 1), two(q.w, 0), two(q.w, 1));
}

// Grid (rows / kReadRows, KV group, sequence).
__global__ void __launch_bounds__(kReadThreads) read_kv8_kernel(ReadArgs a) {
  const int b = blockIdx.z, g = blockIdx.y, tid = threadIdx.x;
  int n = a.n[b];
  if (n > a.max_n) {
    if (tid == 0 && blockIdx.x == 0 && g == 0) flag_status(kStatusClipped);
    n = a.max_n;
  }
  const int i = blockIdx.x * kReadRows + (tid >> 3), lane = tid & 7;
  if (i >= n) return;
  const long long t = (long long)a.start[b] + i;
  const long long lp = t / a.P;
  if (t < 0 || lp >= a.maxp) {
    if (lane == 0) flag_status(kStatusBadToken);
    return;
  }
  const int phys = a.page_table[(size_t)b * a.maxp + lp];
  if (phys < 0 || phys >= a.n_phys) {
    if (lane == 0) flag_status(kStatusBadPage);
    return;
  }
  const size_t row = ((size_t)phys * a.G + g) * a.P + (size_t)(t - lp * a.P);
  const uint4 kq = *reinterpret_cast<const uint4*>(a.k + row * kD + 16 * lane);
  const uint4 vq = *reinterpret_cast<const uint4*>(a.v + row * kD + 16 * lane);
  const uint32_t kx = a.k_exp[row], vx = a.v_exp[row];
  const size_t o = (((size_t)b * a.max_n + i) * a.G + g) * kD + 16 * lane;
  uint4 lo, hi;
  dequantise16(kq, kx, lo, hi);
  reinterpret_cast<uint4*>(a.k_out + o)[0] = lo;
  reinterpret_cast<uint4*>(a.k_out + o)[1] = hi;
  dequantise16(vq, vx, lo, hi);
  reinterpret_cast<uint4*>(a.v_out + o)[0] = lo;
  reinterpret_cast<uint4*>(a.v_out + o)[1] = hi;
}

}  // namespace hhr
