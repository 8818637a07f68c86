// tk_kv8_decode.cuh -- attention of a few query rows over the 8-bit paged
// cache (decode, and a few drafted tokens), and the merge of key ranges.
//
// For sequence b, key/value head h and the rows r = i * G + g (query i of the
// call, query head h * G + g):
//   s_rj = scale q_r . k8_j 2^(ke_j),  O_r = sum_j exp(s_rj - LSE_r) v8_j 2^(ve_j)
// over the visible positions j < vis_r (all of the sequence, or under the
// causal mask up to the row's own position).
//
// Bound by reading the cache once, so the kernel streams it:
//  - Work is the list of (sequence, head, 16-row tile, 64-position unit); every
//    CTA takes an equal run of it, whatever the lengths (they live on the
//    device; each CTA finds its run by a scan over the sequences).  A run that
//    starts or ends inside a segment leaves a partial result (running maximum,
//    sum and unnormalised O in fp32) that a second kernel merges.
//  - A warp takes 16 positions of each unit.  Every lane copies the bytes it
//    will use itself with cp.async into its own slots of a ring, so the loop
//    has no barrier at all.  Which lane takes what is the tensor core's operand
//    layout: the order of a dot product's terms is free, so a lane's 16
//    consecutive bytes of a key row are its operand words of four k-steps; a
//    lane's 16 consecutive values of four positions are, byte-transposed in
//    registers, its operand of all PV steps.
//  - Products are mma.sync m16n8k16 in fp16 with fp32 accumulation: E4M3 is
//    exact in fp16 and one conversion makes two values.  The tensor rate of
//    this path is a quarter of what the stream needs at most (16 rows), so the
//    5th-generation path with its 128-row tiles would gain nothing here.
//
// Numbers: q rows are scaled by a power of two to a largest magnitude in
// [1, 2) before rounding to fp16 (exact but for elements below 2^-14 of the
// row's largest), the factor returning in the fp32 scores.  m (base 2) is the
// running maximum of the scores, l = sum 2^(s - m) in fp32.  O is held
// relative to its own reference M, the running maximum of s + ve, because a
// page's value exponent multiplies its probabilities: P' = 2^(s + ve - M + 6)
// <= 2^14 in fp16 keeps 2^-30 of the largest contribution.  Both references
// move only when exceeded by 2^8, so O is rescaled rarely.
// A NaN code in a masked or stale row must not reach the sums: scores of
// masked positions are replaced, value rows at or past the length are zeroed,
// and where rows of one tile see different positions a NaN among those is
// multiplied for the rows that see it only.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "sm103_ptx.cuh"
#include "tk_device.h"
#include "tk_kv8.h"
#include "tk_kv8_copy.cuh"

namespace tkattn {

struct Kv8AttnParams {
  Kv8Geom g;
  int page_log2;
  const __nv_bfloat16 *q;  // [B, H, Nq, D]
  const uint8_t *k, *v;
  const int8_t *ke, *ve;
  const int *table, *lengths, *counts;  // counts may be null
  __nv_bfloat16 *o;
  float *lse;
  int B, H, G, Nq;  // G = H / Hkv
  int causal;
  float scale_log2;  // scale * log2(e)
  int row_tiles;     // ceil(Nq * G / rows of a tile)
  int ctas;          // runs the work is cut into
  int *err;
  float *part;       // [ctas, 2, rows of a tile, D + 4]
};

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kDecRows = 16;
constexpr int kDecUnit = kDecWarps * 16;  // positions of a unit
constexpr int kDecStages = 4;
constexpr float kDecTau = 8.f;    // lazy references: exceeded by at most 2^8
constexpr float kDecLift = 6.f;   // P' is lifted by 2^6

template <int D>
struct DecCfg {
  static constexpr int kRun = D / 8;            // output columns of a lane's run
  static constexpr int kRunStride = kRun + 4;   // in the merge buffer (bank spread)
  static constexpr int kRowStride = 8 * kRunStride + 4;
  static constexpr int kStageBytes = 16 * D * 2;  // a warp's keys and values of a unit
  static constexpr int kRingBytes = kDecWarps * kDecStages * kStageBytes;
  static constexpr int kMergeBytes = kDecWarps * kDecRows * (kRowStride + 4) * 4;
  static constexpr int kSmem = kRingBytes + kMergeBytes;
};

// A sequence as the kernels use it.
__device__ __forceinline__ int seq_len(const Kv8AttnParams &p, int b, bool *bad) {
  return kv8_length(p.g, p.lengths[b], bad);
}
__device__ __forceinline__ int seq_rows(const Kv8AttnParams &p, int b, bool *bad) {
  if (!p.counts) return p.Nq;
  const int n = p.counts[b];
  if (n < 0 || n > p.Nq) *bad = true;
  return min(max(n, 0), p.Nq);
}
// Units of each of its segments: at least one where it has query rows (a
// sequence without keys still gets its outputs), none where it has not.
__device__ __forceinline__ int seq_units(const Kv8AttnParams &p, int b, int unit) {
  bool bad = false;
  const int rows = seq_rows(p, b, &bad);
  return rows == 0 ? 0 : max(1, (seq_len(p, b, &bad) + unit - 1) / unit);
}

// Positions row i of a sequence sees.
__device__ __forceinline__ int row_sees(const Kv8AttnParams &p, int i, int len, int rows) {
  return p.causal ? max(0, len - (rows - 1 - i)) : len;
}

struct Kv8Place {
  long long total;   // units of the call
  long long prefix;  // units before sequence b
  int b;
};

// Total work, and the sequence in which unit `u` lies (b = B when past the
// end), or with find_b >= 0 the units before sequence find_b.  Whole block;
// ends with a barrier.
__device__ __forceinline__ void kv8_scan(const Kv8AttnParams &p, int unit, long long segs,
                                         long long u_mul, int find_b, Kv8Place *out,
                                         long long *red) {
  const int nthr = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long sum = 0;
  for (int b = threadIdx.x; b < p.B; b += nthr) sum += seq_units(p, b, unit) * segs;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) red[warp] = sum;
  if (threadIdx.x == 0) out->b = p.B;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < nthr / 32; ++w) total += red[w];
  const long long share = max(1LL, (total + p.ctas - 1) / p.ctas);
  const long long u = u_mul * share;
  __syncthreads();
  long long carry = 0;
  for (int base = 0; base < p.B; base += nthr) {
    const int b = base + threadIdx.x;
    const long long v = b < p.B ? seq_units(p, b, unit) * segs : 0;
    long long inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += t;
    }
    if (lane == 31) red[warp] = inc;
    __syncthreads();
    long long before = carry;
    for (int w = 0; w < warp; ++w) before += red[w];
    long long all = carry;
    for (int w = 0; w < nthr / 32; ++w) all += red[w];
    const long long lo = before + inc - v;
    if (b < p.B && (find_b >= 0 ? b == find_b : (u >= lo && u < lo + v))) {
      out->b = b;
      out->prefix = lo;
    }
    carry = all;
    __syncthreads();
  }
  if (threadIdx.x == 0) out->total = total;
  __syncthreads();
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Any byte of w an E4M3 NaN (0x7f or 0xff).
__device__ __forceinline__ bool has_nan4(uint32_t w) {
  return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
}

// Where a run of units stands.
struct DecCursor {
  int b, seg, unit, units, len;
};

__device__ __forceinline__ void dec_advance(const Kv8AttnParams &p, DecCursor &c, int segs) {
  if (++c.unit < c.units) return;
  c.unit = 0;
  if (++c.seg < segs) return;
  c.seg = 0;
  do {
    ++c.b;
  } while (c.b < p.B && (c.units = seq_units(p, c.b, kDecUnit)) == 0);
  if (c.b < p.B) {
    bool bad = false;
    c.len = seq_len(p, c.b, &bad);
  }
}

template <int D>
__global__ void __launch_bounds__(kDecThreads, 2)
    tk_kv8_decode_kernel(const __grid_constant__ Kv8AttnParams p) {
  using C = DecCfg<D>;
  constexpr int kSteps = D / 16;   // k-steps of Q K^T
  constexpr int kChunks = D / 64;  // 16-byte pieces of a key row a lane takes
  constexpr int kTiles = D / 8;    // 8-column tiles of O
  constexpr int kVw = D / 32;      // words of a value row a lane takes
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Kv8Place place;
  __shared__ long long red[kDecWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q8 = lane >> 2, c4 = lane & 3;
  const Kv8Geom &g = p.g;
  const int segs = g.Hkv * p.row_tiles;
  float *merge_o = reinterpret_cast<float *>(smem + C::kRingBytes);
  float *merge_s = merge_o + kDecWarps * kDecRows * C::kRowStride;  // m, M, l of each warp's rows

  if (blockIdx.x == 0) {  // report what is out of range, once
    bool bad = false;
    for (int b = threadIdx.x; b < p.B; b += kDecThreads) {
      seq_len(p, b, &bad);
      seq_rows(p, b, &bad);
    }
    if (bad) atomicCAS(p.err, 0, kDevErrIndex);
  }
  kv8_scan(p, kDecUnit, segs, blockIdx.x, -1, &place, red);
  const long long share = max(1LL, (place.total + p.ctas - 1) / p.ctas);
  const long long u0 = blockIdx.x * share;
  if (u0 >= place.total) return;
  const int nsteps = (int)min(share, place.total - u0);

  DecCursor cons;
  {
    bool bad = false;
    cons.b = place.b;
    cons.units = seq_units(p, cons.b, kDecUnit);
    cons.len = seq_len(p, cons.b, &bad);
    const long long l = u0 - place.prefix;
    cons.seg = (int)(l / cons.units);
    cons.unit = (int)(l % cons.units);
  }
  DecCursor prod = cons;

  const uint32_t ring = smem_addr(smem) + warp * kDecStages * C::kStageBytes;
  // the page of the step that is issued next: an index, -1 no positions
  auto fetch_page = [&]() -> int {
    const int t = prod.unit * kDecUnit + warp * 16;
    return t < prod.len ? p.table[kv8_table_offset(g, prod.b, t >> p.page_log2)] : -2;
  };
  // Copies of one step; the exponents of its page, or bit 16 when there is
  // nothing to read.
  auto issue = [&](int stage, int id) -> int {
    if (!kv8_page_ok(g, id)) {
      if (id != -2 && lane == 0) atomicCAS(p.err, 0, kDevErrIndex);
      cp_async_commit();
      return 1 << 16;
    }
    const int h = prod.seg / p.row_tiles;
    const int t = prod.unit * kDecUnit + warp * 16;
    const long long off = kv8_row_offset(g, id, h, t & (g.page - 1));
    const uint32_t dst = ring + stage * C::kStageBytes;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
        cp_async16(dst + ((n * kChunks + j) * 32 + lane) * 16,
                   p.k + off + (n * 8 + q8) * D + (c4 + 4 * j) * 16);
    const uint32_t dv = dst + 16 * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = 2 * c4 + (i & 1) + (i >> 1) * 8;
      const uint8_t *src = p.v + off + tok * D + q8 * kVw * 4;
      if constexpr (D == 128)
        cp_async16(dv + (i * 32 + lane) * 16, src);
      else
        cp_async8(dv + (i * 32 + lane) * 8, src);
    }
    cp_async_commit();
    const long long eoff = kv8_exp_offset(g, id, h);
    return (int)(uint8_t)p.ke[eoff] | (int)(uint8_t)p.ve[eoff] << 8;
  };

  int ex[kDecStages - 1];
  int next_id = fetch_page();
#pragma unroll
  for (int s = 0; s < kDecStages - 1; ++s) {
    if (s < nsteps) {
      ex[s] = issue(s, next_id);
      dec_advance(p, prod, segs);
      next_id = s + 1 < nsteps ? fetch_page() : -2;
    } else {
      cp_async_commit();
      ex[s] = 1 << 16;
    }
  }

  int step = 0, seg_index = 0;
  while (step < nsteps) {
    // ---------------------------------------------------------- one segment
    const int b = cons.b, h = cons.seg / p.row_tiles;
    const int rt = cons.seg - h * p.row_tiles;
    const int len = cons.len;
    const int n_here = min(cons.units - cons.unit, nsteps - step);
    const bool whole = cons.unit == 0 && n_here == cons.units;
    bool bad = false;
    const int rows = seq_rows(p, b, &bad);
    const int r_end = rows * p.G;
    // this lane's two rows
    int vis[2];
    float f[2];
    uint32_t a[kSteps][4];
    int vis_min = len;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = rt * kDecRows + q8 + 8 * x;
      const int i = r / p.G;
      const bool on = r < r_end;
      vis[x] = on ? row_sees(p, i, len, rows) : 0;
      vis_min = min(vis_min, on ? vis[x] : len);
      const __nv_bfloat16 *src =
          p.q + (((long long)b * p.H + h * p.G + (r - i * p.G)) * p.Nq + i) * D;
      uint2 w[kSteps];
      uint32_t am = 0;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        w[ks] = on ? *reinterpret_cast<const uint2 *>(src + (c4 + 4 * (ks >> 2)) * 16 +
                                                      (ks & 3) * 4)
                   : make_uint2(0, 0);
        am = max_u16x2(am, w[ks].x & 0x7fff7fffu);
        am = max_u16x2(am, w[ks].y & 0x7fff7fffu);
      }
      am = max(am & 0xffffu, am >> 16);
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      int ea = (int)(am >> 7) - 127;
      if (am < 0x80u || am >= 0x7f80u) ea = 0;  // no normal value, or not finite
      ea = max(ea, -126 + 1);
      const float sc = exp2i(-ea < -126 ? -126 : -ea);
      const float back = exp2i(-ea < -126 ? 126 : ea);
      f[x] = p.scale_log2 * back;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        a[ks][x] = bf16x2_to_f16x2_scaled(w[ks].x, sc);
        a[ks][2 + x] = bf16x2_to_f16x2_scaled(w[ks].y, sc);
      }
    }
    vis_min = __reduce_min_sync(0xffffffffu, vis_min);

    float o[kTiles][4];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, mo[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int n = 0; n < n_here; ++n, ++step) {
      // issue the step kDecStages - 1 ahead, then wait for this one's copies
      int ex_new = 1 << 16;
      if (step + kDecStages - 1 < nsteps) {
        ex_new = issue((step + kDecStages - 1) % kDecStages, next_id);
        dec_advance(p, prod, segs);
        next_id = step + kDecStages < nsteps ? fetch_page() : -2;
      } else {
        cp_async_commit();
      }
      cp_async_wait<kDecStages - 1>();
      const int ex_now = ex[0];
#pragma unroll
      for (int s = 0; s + 1 < kDecStages - 1; ++s) ex[s] = ex[s + 1];
      ex[kDecStages - 2] = ex_new;
      const int t0 = (cons.unit + n) * kDecUnit + warp * 16;
      if (ex_now >> 16 || t0 >= len) continue;  // (warp-uniform)
      const uint8_t *st = smem + (warp * kDecStages + step % kDecStages) * C::kStageBytes;
      const float fk = exp2i((int)(int8_t)ex_now);
      const int ev = (int8_t)(ex_now >> 8);

      // S = Q K^T of 16 positions
      float s[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
          const uint4 w =
              *reinterpret_cast<const uint4 *>(st + ((t * kChunks + j) * 32 + lane) * 16);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int ks = 4 * j + i;
            mma_f16(s[t], a[ks][0], a[ks][1], a[ks][2], a[ks][3],
                    e4m3x2_to_f16x2((uint16_t)(ww[i] & 0xffffu)),
                    e4m3x2_to_f16x2((uint16_t)(ww[i] >> 16)));
          }
        }
      }
      const bool edge = t0 + 16 > vis_min;
      float mx[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float fx = f[x] * fk;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float &y = s[t][2 * x + i];
            y *= fx;
            if (edge && t0 + t * 8 + 2 * c4 + i >= vis[x]) y = -INFINITY;
          }
        mx[x] = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1]));
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
      }
      // references, and the factors that moving them takes
      float up[2];
      uint32_t pa[2][2];
      bool moved = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float m_new = mx[x] > m[x] + kDecTau ? mx[x] : m[x];
        const float co = mx[x] + (float)ev;
        const float mo_new = co > mo[x] + kDecTau ? co : mo[x];
        l[x] *= m_new == m[x] ? 1.f : ex2_approx(m[x] - m_new);
        up[x] = mo_new == mo[x] ? 1.f : ex2_approx(mo[x] - mo_new);
        moved |= mo_new != mo[x];
        m[x] = m_new;
        mo[x] = mo_new;
        const float mu = m_new == -INFINITY ? 0.f : m_new;
        // P = 2^(s - m), P' = P 2^(m + ve - M + 6)
        const float lift =
            ex2_approx(fminf((m_new == -INFINITY ? -200.f : m_new + (float)ev - mo_new) + kDecLift,
                             120.f));
        float pr[4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float e = ex2_approx(s[t][2 * x + i] - mu);
            l[x] += e;
            pr[2 * t + i] = e * lift;
          }
        pa[0][x] = pack_f16x2(pr[0], pr[1]);
        pa[1][x] = pack_f16x2(pr[2], pr[3]);
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          o[j][0] *= up[0];
          o[j][1] *= up[0];
          o[j][2] *= up[1];
          o[j][3] *= up[1];
        }
      }
      // O += P' V
      uint32_t w[4][kVw];
      const uint8_t *sv = st + 16 * D;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128) {
          const uint4 y = *reinterpret_cast<const uint4 *>(sv + (i * 32 + lane) * 16);
          w[i][0] = y.x;
          w[i][1] = y.y;
          w[i][2] = y.z;
          w[i][3] = y.w;
        } else {
          const uint2 y = *reinterpret_cast<const uint2 *>(sv + (i * 32 + lane) * 8);
          w[i][0] = y.x;
          w[i][1] = y.y;
        }
      }
      int i_lo = 0, i_hi = 0;  // rows in one go, or query by query
      if (edge) {
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = t0 + 2 * c4 + (i & 1) + (i >> 1) * 8;
#pragma unroll
          for (int y = 0; y < kVw; ++y) {
            if (tok >= len) w[i][y] = 0;
            odd |= tok >= vis_min && has_nan4(w[i][y]);
          }
        }
        if (__any_sync(0xffffffffu, odd)) {
          i_lo = rt * kDecRows / p.G;
          i_hi = min(rows - 1, (rt * kDecRows + kDecRows - 1) / p.G);
          for (int i = i_lo; i <= i_hi; ++i) {
            const int see = row_sees(p, i, len, rows);
            const int ra = rt * kDecRows + q8;
            const bool on0 = ra / p.G == i, on1 = (ra + 8) / p.G == i;
            uint32_t z[4][kVw];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int y = 0; y < kVw; ++y)
                z[k][y] = t0 + 2 * c4 + (k & 1) + (k >> 1) * 8 < see ? w[k][y] : 0u;
#pragma unroll
            for (int y = 0; y < kVw; ++y)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t sel = half ? 0x7362 : 0x5140;
                const uint32_t x0 = __byte_perm(z[0][y], z[1][y], sel);
                const uint32_t x1 = __byte_perm(z[2][y], z[3][y], sel);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  float t[4] = {0.f, 0.f, 0.f, 0.f};
                  mma_f16(t, pa[0][0], pa[0][1], pa[1][0], pa[1][1],
                          e4m3x2_to_f16x2((uint16_t)(x0 >> (16 * k))),
                          e4m3x2_to_f16x2((uint16_t)(x1 >> (16 * k))));
                  float(&oo)[4] = o[4 * y + 2 * half + k];
                  if (on0) {
                    oo[0] += t[0];
                    oo[1] += t[1];
                  }
                  if (on1) {
                    oo[2] += t[2];
                    oo[3] += t[3];
                  }
                }
              }
          }
          continue;
        }
      }
#pragma unroll
      for (int y = 0; y < kVw; ++y)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? 0x7362 : 0x5140;
          const uint32_t x0 = __byte_perm(w[0][y], w[1][y], sel);
          const uint32_t x1 = __byte_perm(w[2][y], w[3][y], sel);
          mma_f16(o[4 * y + 2 * half], pa[0][0], pa[0][1], pa[1][0], pa[1][1],
                  e4m3x2_to_f16x2((uint16_t)(x0 & 0xffffu)),
                  e4m3x2_to_f16x2((uint16_t)(x1 & 0xffffu)));
          mma_f16(o[4 * y + 2 * half + 1], pa[0][0], pa[0][1], pa[1][0], pa[1][1],
                  e4m3x2_to_f16x2((uint16_t)(x0 >> 16)), e4m3x2_to_f16x2((uint16_t)(x1 >> 16)));
        }
    }

    // ---------------------------------------------------------- join the warps
    __syncthreads();  // the merge buffer is free
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      const int row = q8 + 8 * x;
      if (c4 == 0) {
        float *d = merge_s + (warp * kDecRows + row) * 4;
        d[0] = m[x];
        d[1] = mo[x];
        d[2] = l[x];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float *d = merge_o + (warp * kDecRows + row) * C::kRowStride + (2 * c4 + i) * C::kRunStride;
#pragma unroll
        for (int j = 0; j < kTiles; j += 4)
          *reinterpret_cast<float4 *>(d + j) =
              make_float4(o[j][2 * x + i], o[j + 1][2 * x + i], o[j + 2][2 * x + i],
                          o[j + 3][2 * x + i]);
      }
    }
    __syncthreads();
    {
      const int row = threadIdx.x >> 3, run = threadIdx.x & 7;
      const int r = rt * kDecRows + row;
      if (r < r_end) {
        float mm = -INFINITY, mmo = -INFINITY, ll = 0.f;
        float wt[kDecWarps];
#pragma unroll
        for (int w2 = 0; w2 < kDecWarps; ++w2) {
          const float *d = merge_s + (w2 * kDecRows + row) * 4;
          mm = fmaxf(mm, d[0]);
          mmo = fmaxf(mmo, d[1]);
        }
#pragma unroll
        for (int w2 = 0; w2 < kDecWarps; ++w2) {
          const float *d = merge_s + (w2 * kDecRows + row) * 4;
          // nothing seen: l is 0 (a NaN score leaves l NaN, which has to stay)
          ll += d[2] == 0.f ? 0.f : d[2] * ex2_approx(d[0] - mm);
          wt[w2] = d[2] == 0.f ? 0.f : ex2_approx(d[1] - mmo);
        }
        float out[C::kRun];
#pragma unroll
        for (int j = 0; j < C::kRun; ++j) out[j] = 0.f;
#pragma unroll
        for (int w2 = 0; w2 < kDecWarps; ++w2) {
          const float *d = merge_o + (w2 * kDecRows + row) * C::kRowStride + run * C::kRunStride;
#pragma unroll
          for (int j = 0; j < C::kRun; j += 4) {
            const float4 y = *reinterpret_cast<const float4 *>(d + j);
            out[j] = fmaf(wt[w2], y.x, out[j]);
            out[j + 1] = fmaf(wt[w2], y.y, out[j + 1]);
            out[j + 2] = fmaf(wt[w2], y.z, out[j + 2]);
            out[j + 3] = fmaf(wt[w2], y.w, out[j + 3]);
          }
        }
        if (whole) {
          const int i = r / p.G;
          const long long orow = ((long long)b * p.H + h * p.G + (r - i * p.G)) * p.Nq + i;
          // 2^(M - 6 - m) / l, in two factors (M - m is a value exponent)
          const float half = ll == 0.f ? 0.f : ex2_approx(0.5f * (mmo - kDecLift - mm));
          const float inv = ll == 0.f ? 0.f : half / ll;
          uint32_t pk[C::kRun / 2];
#pragma unroll
          for (int j = 0; j < C::kRun / 2; ++j)
            pk[j] = pack_bf16x2(out[2 * j] * inv * half, out[2 * j + 1] * inv * half);
          uint4 *dst = reinterpret_cast<uint4 *>(p.o + orow * D + run * C::kRun);
#pragma unroll
          for (int j = 0; j < C::kRun / 8; ++j)
            dst[j] = make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
          if (run == 0)
            p.lse[orow] =
                ll == 0.f ? -INFINITY : (mm + lg2_approx(ll)) * 0.69314718055994531f;
        } else {
          float *d = p.part + (((size_t)blockIdx.x * 2 + (seg_index > 0)) * kDecRows + row) *
                                  (D + 4);
#pragma unroll
          for (int j = 0; j < C::kRun; j += 4)
            *reinterpret_cast<float4 *>(d + run * C::kRun + j) =
                make_float4(out[j], out[j + 1], out[j + 2], out[j + 3]);
          if (run == 0) *reinterpret_cast<float4 *>(d + D) = make_float4(mm, mmo, ll, 0.f);
        }
      }
    }
    // next segment
    ++seg_index;
    cons.unit += n_here - 1;
    dec_advance(p, cons, segs);
  }
}

// Merge of the runs' partial results: one block (a thread a column) for each
// (head and row tile, sequence, row).  Segments that one run held whole are
// already written.
template <int D>
__global__ void __launch_bounds__(D)
    tk_kv8_merge_kernel(const __grid_constant__ Kv8AttnParams p) {
  __shared__ Kv8Place place;
  __shared__ long long red[4];
  const int seg = blockIdx.x, b = blockIdx.y, row = blockIdx.z;
  const int segs = p.g.Hkv * p.row_tiles;
  const int h = seg / p.row_tiles, rt = seg - h * p.row_tiles;
  bool bad = false;
  const int rows = seq_rows(p, b, &bad);
  const int r = rt * kDecRows + row;
  if (r >= rows * p.G) return;
  kv8_scan(p, kDecUnit, segs, 0, b, &place, red);
  const int units = seq_units(p, b, kDecUnit);
  const long long share = max(1LL, (place.total + p.ctas - 1) / p.ctas);
  const long long s0 = place.prefix + (long long)seg * units;
  const int c0 = (int)(s0 / share), c1 = (int)((s0 + units - 1) / share);
  if (c0 == c1) return;
  // run c0's partial is its first segment's only if it starts where the segment does
  const float *base = p.part + (size_t)row * (D + 4);
  const size_t slot = (size_t)kDecRows * (D + 4);
  const int first0 = c0 * share == s0 ? 0 : 1;
  auto at = [&](int c) { return base + ((size_t)c * 2 + (c == c0 ? first0 : 0)) * slot; };
  float mm = -INFINITY, mmo = -INFINITY;
  for (int c = c0; c <= c1; ++c) {
    mm = fmaxf(mm, at(c)[D]);
    mmo = fmaxf(mmo, at(c)[D + 1]);
  }
  float ll = 0.f, out = 0.f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const float *d = at(c);
    const float l = d[D + 2];
    ll += l == 0.f ? 0.f : l * ex2_approx(d[D] - mm);
    out = fmaf(l == 0.f ? 0.f : ex2_approx(d[D + 1] - mmo), d[threadIdx.x], out);
  }
  const int i = r / p.G;
  const long long orow = ((long long)b * p.H + h * p.G + (r - i * p.G)) * p.Nq + i;
  const float half = ll == 0.f ? 0.f : ex2_approx(0.5f * (mmo - kDecLift - mm));
  const float inv = ll == 0.f ? 0.f : half / ll;
  p.o[orow * D + threadIdx.x] = __float2bfloat16(out * inv * half);
  if (threadIdx.x == 0)
    p.lse[orow] = ll == 0.f ? -INFINITY : (mm + lg2_approx(ll)) * 0.69314718055994531f;
}

}  // namespace tkattn
