// tk_kv8_copy.cuh -- writing keys and values into the 8-bit paged cache and
// reading them back.
//
// Write: a block owns one (page, head) of one of the two payloads, so the
// page's exponent and rows have one writer.  It reads the page's new rows
// once (16 bytes a load, kept in registers), takes their largest magnitude
// with packed integer maxima on the bf16 bits, settles the exponent
//   e = max(least e with 448 * 2^e >= magnitude, exponent held if rows before
//       the write stay),
// rounds x * 2^-e to E4M3 (the scaling is exact, so the rounding is the only
// one) and, when e grew, rounds the rows that stay again: code * 2^(old - e).
// NaN and infinite inputs become E4M3's NaN and do not enter the exponent.
//
// Read: payload -> fp16 (exact) -> fp32, times 2^e (exact), -> bf16 (exact for
// the exponents a write gives).
// Both are bound by the bytes they move.  Measured, with 8 heads of 128: up to
// 4096 tokens written for each of 8 sequences in 18.6 us (114 MB, 6.1 TB/s); one
// for each of 64 in 4.0 us, most of it the start of a grid and three dependent
// reads (position, page, exponent); 8 sequences of up to 16384 positions read
// back in 72 us (453 MB, 6.3 TB/s).
// A write's block is a page, not more, because a page's exponent needs all of
// its new rows; its thread keeps kPage / 128 * D / 8 loads in flight, so a
// kernel for each page size holds no more registers than its page needs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "sm103_ptx.cuh"
#include "tk_device.h"
#include "tk_kv8.h"
#include "tk_launch.cuh"

namespace tkattn {

constexpr int kKv8Threads = 128;

struct Kv8WriteParams {
  Kv8Geom g;
  const __nv_bfloat16 *src[2];  // new keys, new values
  long long sb[2], sh[2], sn[2];
  uint8_t *payload[2];
  int8_t *exps[2];
  const int *table, *start, *counts;  // counts may be null (every row counts)
  int B, N;
  int early;  // the next grid may begin beside this one (tk_launch.cuh)
  int *err;
};

// Two fp32 -> two E4M3 codes (round to nearest even), `lo` in bits 0-7.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two E4M3 codes -> f16x2 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t v) {
  const uint32_t h = e4m3x2_to_f16x2(v);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Four bf16 values times 2^-e, to four codes.
__device__ __forceinline__ uint32_t quant4(uint32_t v, uint32_t w, float s) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(__uint_as_float(v << 16) * s), "f"(__uint_as_float(v & 0xffff0000u) * s),
        "f"(__uint_as_float(w << 16) * s), "f"(__uint_as_float(w & 0xffff0000u) * s));
  return r;
}

// Infinities of a bf16x2 to NaN (E4M3 has none, and the conversion would make
// them the largest value).
__device__ __forceinline__ uint32_t inf_to_nan(uint32_t v) {
  if ((v & 0x7fffu) == 0x7f80u) v |= 0x40u;
  if ((v & 0x7fff0000u) == 0x7f800000u) v |= 0x400000u;
  return v;
}

// Largest finite magnitude of a bf16x2's two halves, as bits.
__device__ __forceinline__ uint32_t finite_max(uint32_t v) {
  const uint32_t a = v & 0x7fffu, b = (v >> 16) & 0x7fffu;
  return max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u);
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *red) {
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();  // red free
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t m = red[0];
#pragma unroll
  for (int i = 1; i < kKv8Threads / 32; ++i) m = max(m, red[i]);
  return m;
}

// grid: (pages a write can touch, 2 * Hkv, B)
template <int D, int kPage>
__global__ void __launch_bounds__(kKv8Threads)
    tk_kv8_write_kernel(const __grid_constant__ Kv8WriteParams p) {
  constexpr int kVec = D / 8;                          // 16-byte loads a row
  constexpr int kMaxVec = kPage * kVec / kKv8Threads;  // a thread's loads of a whole page
  constexpr int kRowsStep = kKv8Threads / kVec;        // rows from one of them to the next
  __shared__ uint32_t red[kKv8Threads / 32];
  const Kv8Geom &g = p.g;
  const int b = blockIdx.z;
  const int which = blockIdx.y >= g.Hkv;
  const int h = blockIdx.y - (which ? g.Hkv : 0);
  grid_launch_dependents_if(p.early);
  grid_wait();
  bool bad = false;
  const int start = p.start[b];
  const int n = kv8_write_rows(g, start, p.counts ? p.counts[b] : p.N, p.N, &bad);
  if (bad && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    atomicCAS(p.err, 0, kDevErrIndex);
  if (n == 0) return;
  const int slot = start / kPage + blockIdx.x;
  const long long at = (long long)slot * kPage;
  if (at >= start + n) return;
  const int first = (int)at;                // position of the page's row 0
  const int r0 = max(start - first, 0);     // the page's new rows are [r0, r1)
  const int r1 = min(start + n - first, kPage);
  const int id = p.table[kv8_table_offset(g, b, slot)];
  // the new rows, in registers
  const int row = threadIdx.x / kVec, col = threadIdx.x % kVec;  // this thread's first piece
  const long long step = kRowsStep * p.sn[which];
  const __nv_bfloat16 *src = p.src[which] + b * p.sb[which] + h * p.sh[which] +
                             (long long)(first + r0 - start + row) * p.sn[which] + col * 8;
  const int rows = r1 - r0;
  uint4 v[kMaxVec];
#pragma unroll
  for (int i = 0; i < kMaxVec; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    if (row + i * kRowsStep < rows) v[i] = __ldg(reinterpret_cast<const uint4 *>(src));
    src += step;
  }
  if (!kv8_page_ok(g, id)) {
    if (threadIdx.x == 0) atomicCAS(p.err, 0, kDevErrIndex);
    return;
  }
  const long long eoff = kv8_exp_offset(g, id, h);
  const int held = r0 > 0 ? p.exps[which][eoff] : -128;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kMaxVec; ++i) {
    m = max_u16x2(m, v[i].x & 0x7fff7fffu);
    m = max_u16x2(m, v[i].y & 0x7fff7fffu);
    m = max_u16x2(m, v[i].z & 0x7fff7fffu);
    m = max_u16x2(m, v[i].w & 0x7fff7fffu);
  }
  m = block_max(max(m & 0xffffu, m >> 16), red);
  const bool odd = m >= 0x7f80u;  // a NaN or an infinity among the rows: leave it out
  if (odd) {
    m = 0;
#pragma unroll
    for (int i = 0; i < kMaxVec; ++i)
      m = max(max(max(m, finite_max(v[i].x)), finite_max(v[i].y)),
              max(finite_max(v[i].z), finite_max(v[i].w)));
    m = block_max(m, red);
  }
  const int e = max(kv8_exponent(m), held);
  uint8_t *page = p.payload[which] + kv8_row_offset(g, id, h, 0);
  if (threadIdx.x == 0) p.exps[which][eoff] = (int8_t)e;
  if (held > -128 && e > held) {
    // rows that stay, onto the new grid
    const float s = exp2i(max(held - e, -126));
    uint2 *old = reinterpret_cast<uint2 *>(page);
    constexpr int kDeep = kMaxVec < 4 ? kMaxVec : 4;  // reads in flight
#pragma unroll 1
    for (int c0 = threadIdx.x; c0 < r0 * kVec; c0 += kDeep * kKv8Threads) {
      uint2 w[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u)
        if (c0 + u * kKv8Threads < r0 * kVec) w[u] = old[c0 + u * kKv8Threads];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        if (c0 + u * kKv8Threads >= r0 * kVec) break;
        uint32_t *q = reinterpret_cast<uint32_t *>(&w[u]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 a = e4m3x2_to_float2((uint16_t)(q[i] & 0xffffu));
          const float2 c2 = e4m3x2_to_float2((uint16_t)(q[i] >> 16));
          q[i] = pack_e4m3x2(a.x * s, a.y * s) | pack_e4m3x2(c2.x * s, c2.y * s) << 16;
        }
        old[c0 + u * kKv8Threads] = w[u];
      }
    }
  }
  const float s = exp2i(max(-e, -126));
  uint2 *dst = reinterpret_cast<uint2 *>(page + r0 * D) + threadIdx.x;
  if (odd) {  // infinities become NaN before the scaling
#pragma unroll
    for (int i = 0; i < kMaxVec; ++i) {
      v[i].x = inf_to_nan(v[i].x);
      v[i].y = inf_to_nan(v[i].y);
      v[i].z = inf_to_nan(v[i].z);
      v[i].w = inf_to_nan(v[i].w);
    }
  }
#pragma unroll
  for (int i = 0; i < kMaxVec; ++i)
    if (row + i * kRowsStep < rows)
      dst[i * kKv8Threads] =
          make_uint2(quant4(v[i].x, v[i].y, s), quant4(v[i].z, v[i].w, s));
}

struct Kv8ReadParams {
  Kv8Geom g;
  const uint8_t *payload[2];
  const int8_t *exps[2];
  const int *table, *lengths;
  __nv_bfloat16 *dst[2];  // [B, Hkv, N, D]
  int B, N;
  int early;  // the next grid may begin beside this one (tk_launch.cuh)
  int *err;
};

// grid: (ceil(N / 64), 2 * Hkv, B); a block reads 64 positions of one head.
template <int D>
__global__ void __launch_bounds__(kKv8Threads)
    tk_kv8_read_kernel(const __grid_constant__ Kv8ReadParams p) {
  constexpr int kVec = D / 16;  // 16-byte loads a row
  constexpr int kPer = 64 * kVec / kKv8Threads;
  const Kv8Geom &g = p.g;
  const int b = blockIdx.z;
  const int which = blockIdx.y >= g.Hkv;
  const int h = blockIdx.y - (which ? g.Hkv : 0);
  grid_launch_dependents_if(p.early);
  grid_wait();
  bool bad = false;
  const int len = kv8_length(g, p.lengths[b], &bad);
  if (bad && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    atomicCAS(p.err, 0, kDevErrIndex);
  const int rows = min(len, p.N);
  const int t0 = blockIdx.x * 64;
  if (t0 >= rows) return;
  uint4 v[kPer];
  int e[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = threadIdx.x + i * kKv8Threads;
    const int t = t0 + c / kVec;
    e[i] = 128;  // no row
    v[i] = make_uint4(0, 0, 0, 0);
    if (t < rows) {
      const int id = p.table[kv8_table_offset(g, b, t / g.page)];
      if (kv8_page_ok(g, id)) {
        v[i] = *reinterpret_cast<const uint4 *>(p.payload[which] +
                                                kv8_row_offset(g, id, h, t % g.page) +
                                                (c % kVec) * 16);
        e[i] = p.exps[which][kv8_exp_offset(g, id, h)];
      } else {
        atomicCAS(p.err, 0, kDevErrIndex);
      }
    }
  }
  __nv_bfloat16 *dst = p.dst[which] + (((long long)b * g.Hkv + h) * p.N + t0) * D;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (e[i] == 128) continue;
    const int c = threadIdx.x + i * kKv8Threads;
    // 2^e in two exact factors, for exponents at the ends of the range
    const float s0 = exp2i(e[i] / 2), s1 = exp2i(e[i] - e[i] / 2);
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = e4m3x2_to_float2((uint16_t)(w[j] & 0xffffu));
      const float2 d = e4m3x2_to_float2((uint16_t)(w[j] >> 16));
      o[2 * j] = pack_bf16x2(a.x * s0 * s1, a.y * s0 * s1);
      o[2 * j + 1] = pack_bf16x2(d.x * s0 * s1, d.y * s0 * s1);
    }
    uint4 *out = reinterpret_cast<uint4 *>(dst + (c / kVec) * D + (c % kVec) * 16);
    out[0] = make_uint4(o[0], o[1], o[2], o[3]);
    out[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace tkattn
