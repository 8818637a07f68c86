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
//  - Work is the list of (sequence, head, 64-position unit); every
//    CTA takes an equal run of it, whatever the lengths (they live on the
//    device; each CTA finds its run by a scan over the sequences).  A run that
//    starts or ends inside a segment leaves a partial result (running maximum,
//    sum and unnormalised O in fp32) that a second kernel merges.
//  - A warp takes 16 positions of each unit, 16 D bytes of keys and as many of
//    values (a page is a multiple of 16 positions), copied by cp.async
//    into its own ring: no barrier but the warp's own.  Rows are stored with
//    their 16-byte pieces exchanged so that the operand loads are free of bank
//    conflicts.  The order of a dot product's terms is free, so a lane's 16
//    consecutive bytes of a key row are its operand words of four k-steps; a
//    lane's D/8 consecutive values of four positions are, byte-transposed in
//    registers, its operand of all PV steps.  (Copies in which a lane fetched
//    what it would use, half a line a row, brought every line of keys twice
//    from L2: 5.0 TB/s.)
//  - Products are mma.sync m16n8k16 in fp16 with fp32 accumulation, positions
//    (S^T = K Q^T) and value columns (O^T = V^T P^T) on the 16-row side, query
//    rows on the 8-wide side: E4M3 is exact in fp16, one conversion makes two
//    values, and eight rows fill a tile.  With the query rows on the 16-row
//    side the same step took twice the products, exponentials and accumulators:
//    232 registers, two warps a scheduler, 3.8 TB/s at 8 x 16384 positions of
//    32 heads.  The 5th-generation path has 128-row tiles, sixteen times the
//    rows there are.
//
// Measured: one query for each of 8 sequences of 16384 positions and 32 heads of
// 128, 159 us, 6.76 TB/s (the rate of a plain copy); 32 sequences of up to 32768
// positions, 4 query heads a key head, 164 us, 6.74 TB/s; one sequence of 1000
// positions 6.0 us, most of it the start of two grids and four dependent reads
// (length, page, codes, partials).  With 40 rows (5 drafts, 8 heads a key head, D = 64) the
// products, exponentials and conversions bound it: 33.7 us for what a copy reads
// in 5.4, the eight warps that an SM's registers hold issuing 40 % of the time.
//
// Numbers: q rows are scaled by a power of two to a largest magnitude in
// [1, 2) before rounding to fp16 (exact but for elements below 2^-14 of the
// row's largest), the factor returning in the fp32 scores.  m (base 2) is the
// running maximum of the scores, moved only when a score exceeds it by 2^8;
// l = sum 2^(s - m) in fp32.  A page's value exponent multiplies its
// probabilities, so O is held relative to its own reference M, the running
// maximum of m + ve: P' = 2^(s + ve - M + 7) <= 2^15 in fp16, whose least value
// is 2^-31 of a weight 1 in the page of the largest exponent.  While neither
// reference moves, a step has no exchange between lanes but the operand's
// transposition and one vote.
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
#include "tk_launch.cuh"

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
  unsigned g_mul;   // floor(2^32 / G) + 1, or 0 for G = 1
  int causal;
  float scale_log2;  // scale * log2(e)
  int tile_rows;     // (few rows) a tile's rows, at least Nq * G
  int pair;          // (many rows) the two tiles of a unit share its rows
  int ctas;          // runs the work is cut into
  int *err;
  float *part;       // [ctas, 2, rows of a tile or unit, D + 4]
  long long *prefix;  // (many rows) the work before each sequence, a run's share last
};

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kDecUnit = kDecWarps * 16;  // positions of a unit
constexpr float kDecTau = 8.f;       // m is exceeded by at most 2^8
constexpr float kDecLift = 7.f;      // P' is lifted by 2^7
constexpr float kDecNone = -1e30f;   // references before any score
constexpr float kDecNoLift = -200.f;  // and what lifts P' then (no value exponent makes it large)

// kNT tiles of eight query rows a warp: up to 40 rows at D = 64 and 24 at
// D = 128, where the accumulators (kNT * D / 4 a thread) still fit the registers.
// From three tiles on, the queries' operands come from shared memory.
template <int D, int kNT>
struct DecCfg {
  static constexpr int kRows = 8 * kNT;
  static constexpr int kStages = 3;
  static constexpr int kRun = D / 8;            // output columns of a lane's run
  static constexpr int kRunStride = kRun + 4;   // in the merge buffer (bank spread)
  static constexpr int kRowStride = 8 * kRunStride + 4;
  static constexpr int kStageBytes = 16 * D * 2;  // a warp's keys and values of a unit
  static constexpr int kRingBytes = kDecWarps * kStages * kStageBytes;
  // the warps' parts of kJoin tiles of eight rows, and their statistics
  static constexpr int kJoin = D == 128 && kNT > 2 ? 2 : kNT;
  static constexpr int kMergeRows = 8 * kJoin;
  static constexpr int kMergeBytes = kDecWarps * kMergeRows * (kRowStride + 4) * 4;
  static constexpr bool kQShared = kNT > 2;
  static constexpr int kQBytes = kQShared ? kRows * (D * 2 + 4) : 0;  // operands, factors
  static constexpr int kSmem = kRingBytes + kMergeBytes + kQBytes;
  static constexpr int kCtasPerSm = D == 64 ? (kNT <= 1 ? 4 : kNT <= 3 ? 3 : 2) : (kNT == 1 ? 3 : 2);
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

// Query of row r = i * G + g (the host bounds Nq * G * G below 2^31, which makes
// the multiplication exact).
__device__ __forceinline__ int row_query(const Kv8AttnParams &p, int r) {
  return p.g_mul ? (int)__umulhi((unsigned)r, p.g_mul) : r;
}
// Positions row i of a sequence sees.
__device__ __forceinline__ int row_sees(const Kv8AttnParams &p, int i, int len, int rows) {
  return p.causal ? max(0, len - (rows - 1 - i)) : len;
}

struct Kv8Place {
  long long total;   // units of the call
  long long share;   // units of a run
  long long prefix;  // units before sequence b
  int b;
};

// Total work (cost(b) over the sequences), and the sequence in which run `run`
// starts (b = B when past the end).  With `prefix` the work before each sequence is written
// there, a run's share last.  Whole block; ends with a barrier.
template <typename Cost>
__device__ __forceinline__ void kv8_scan(const Kv8AttnParams &p, Cost cost, int run, Kv8Place *out,
                                         long long *red, long long *prefix) {
  const int nthr = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long v0 = (int)threadIdx.x < p.B ? cost(threadIdx.x) : 0;
  long long sum = v0;
#pragma unroll 1
  for (int b = threadIdx.x + nthr; b < p.B; b += nthr) sum += cost(b);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) red[warp] = sum;
  if (threadIdx.x == 0) out->b = p.B;
  __syncthreads();
  long long total = 0;
#pragma unroll 1
  for (int w = 0; w < nthr / 32; ++w) total += red[w];
  if (threadIdx.x == 0) {
    const long long share = max(1LL, (total + p.ctas - 1) / p.ctas);
    out->total = total;
    out->share = share;
    if (prefix) prefix[p.B] = share;
  }
  __syncthreads();
  const long long u = run * out->share;
  long long carry = 0;
#pragma unroll 1
  for (int base = 0; base < p.B; base += nthr) {
    const int b = base + threadIdx.x;
    const long long v = base == 0 ? v0 : b < p.B ? cost(b) : 0;
    long long inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += t;
    }
    if (lane == 31) red[warp] = inc;
    __syncthreads();
    long long before = carry;
#pragma unroll 1
    for (int w = 0; w < nthr / 32; ++w) {
      const long long x = red[w];
      before += w < warp ? x : 0;
      carry += x;
    }
    const long long lo = before + inc - v;
    if (b < p.B) {
      if (prefix) prefix[b] = lo;
      if (u >= lo && u < lo + v) {
        out->b = b;
        out->prefix = lo;
      }
    }
    __syncthreads();
  }
}

// The same for few rows, in 32 bits (the host bounds the units) and with one
// value a thread in hand: total work, and where run `run` starts.  Two barriers
// for up to kDecThreads sequences.
struct DecPlace {
  int total, share, b, prefix;
};
__device__ __forceinline__ void dec_scan(const Kv8AttnParams &p, int run, DecPlace *out,
                                         int (*red)[kDecWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int v0 = (int)threadIdx.x < p.B ? seq_units(p, threadIdx.x, kDecUnit) * p.g.Hkv : 0;
  int sum = v0, inc = v0;
#pragma unroll 1
  for (int b = threadIdx.x + kDecThreads; b < p.B; b += kDecThreads)
    sum += seq_units(p, b, kDecUnit) * p.g.Hkv;
  sum = __reduce_add_sync(0xffffffffu, sum);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += t;
  }
  if (lane == 31) {
    red[0][warp] = sum;
    red[1][warp] = inc;
  }
  __syncthreads();
  int total = 0, lo = inc - v0, all = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    total += red[0][w];
    if (w < warp) lo += red[1][w];
    all += red[1][w];
  }
  const int share = max(1, (int)(((unsigned)total + p.ctas - 1) / (unsigned)p.ctas));
  const int u = run * share;  // (at most the total and a share)
  if (threadIdx.x == 0) {
    out->total = total;
    out->share = share;
  }
  if (u >= lo && u < lo + v0) {
    out->b = threadIdx.x;
    out->prefix = lo;
  }
#pragma unroll 1
  for (int base = kDecThreads; base < p.B && all <= u; base += kDecThreads) {
    // more sequences than threads: on to the next kDecThreads of them
    const int b = base + threadIdx.x;
    const int v = b < p.B ? seq_units(p, b, kDecUnit) * p.g.Hkv : 0;
    inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += t;
    }
    __syncthreads();
    if (lane == 31) red[1][warp] = inc;
    __syncthreads();
    lo = all + inc - v;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      if (w < warp) lo += red[1][w];
      all += red[1][w];
    }
    if (u >= lo && u < lo + v) {
      out->b = b;
      out->prefix = lo;
    }
  }
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
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// An 8 x 8 matrix of 16-bit values, one row to four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Four E4M3 codes -> two f16x2 (bytes 0, 1 and 2, 3).
__device__ __forceinline__ void e4m3x4_to_f16x2x2(uint32_t w, uint32_t &a, uint32_t &b) {
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(w));
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

template <int D, int kNT>
__global__ void __launch_bounds__(kDecThreads, DecCfg<D, kNT>::kCtasPerSm)
    tk_kv8_decode_kernel(const __grid_constant__ Kv8AttnParams p) {
  using C = DecCfg<D, kNT>;
  constexpr int kStages = C::kStages;
  constexpr int kSteps = D / 16;   // k-steps of K Q^T, 16-column tiles of O
  constexpr int kChunks = D / 64;  // 16-byte pieces of a key row a lane takes
  constexpr int kVw = D / 32;      // words of a value row a lane takes
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ DecPlace place;
  __shared__ int red[2][kDecWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q8 = lane >> 2, c4 = lane & 3;
  const Kv8Geom &g = p.g;
  const int segs = g.Hkv;  // segments of a sequence
  float *merge_o = reinterpret_cast<float *>(smem + C::kRingBytes);
  float *merge_s = merge_o + kDecWarps * C::kMergeRows * C::kRowStride;  // m, M, l of each warp's rows
  uint4 *q_ops = reinterpret_cast<uint4 *>(smem + C::kRingBytes + C::kMergeBytes);
  float *q_fac = reinterpret_cast<float *>(q_ops + kNT * (kSteps / 2) * 32);  // of each row

  grid_wait();
  grid_launch_dependents();  // (after the wait: the merge reads the lengths before its own)
  if (blockIdx.x == 0) {  // report what is out of range, once
    bool bad = false;
#pragma unroll 1
    for (int b = threadIdx.x; b < p.B; b += kDecThreads) {
      seq_len(p, b, &bad);
      seq_rows(p, b, &bad);
    }
    if (bad) atomicCAS(p.err, 0, kDevErrIndex);
  }
  dec_scan(p, blockIdx.x, &place, red);
  const int u0 = blockIdx.x * place.share;
  if (u0 >= place.total) return;
  const int nsteps = min(place.share, place.total - u0);

  DecCursor cons;
  {
    bool bad = false;
    cons.b = place.b;
    cons.units = seq_units(p, cons.b, kDecUnit);
    cons.len = seq_len(p, cons.b, &bad);
    cons.seg = (u0 - place.prefix) / cons.units;
    cons.unit = u0 - place.prefix - cons.seg * cons.units;
  }
  DecCursor prod = cons;

  // this lane's places in 16 rows: the copies' destination, and the operand
  // reads' (rows of 128 bytes: piece ^ row % 8; of 64 bytes: piece ^ row / 2 % 4)
  uint32_t put, k_get, v_get[2];
  if constexpr (D == 128) {
    put = (lane >> 3) * 128 + ((lane & 7) ^ (lane >> 3)) * 16;
    k_get = q8 * 128 + ((2 * c4) ^ q8) * 16;  // piece 2 c4 + j: ^ 16 j
    v_get[0] = (2 * c4) * 128 + (q8 ^ (2 * c4)) * 16;
    v_get[1] = (2 * c4 + 1) * 128 + (q8 ^ (2 * c4 + 1)) * 16;
  } else {
    put = (lane >> 2) * 64 + ((lane & 3) ^ ((lane >> 3) & 3)) * 16;
    k_get = q8 * 64 + (c4 ^ (q8 >> 1)) * 16;
    v_get[0] = (2 * c4) * 64 + ((q8 >> 1) ^ c4) * 16 + (q8 & 1) * 8;
    v_get[1] = v_get[0] + 64;
  }
  const uint32_t ring = smem_addr(smem) + warp * kStages * C::kStageBytes + put;
  // the page of the step that is issued next: an index, -2 no positions
  auto fetch_page = [&]() -> int {
    const int t = prod.unit * kDecUnit + warp * 16;
    return t < prod.len ? p.table[kv8_table_offset(g, prod.b, t >> p.page_log2)] : -2;
  };
  // Copies of one step; where its page's exponents lie, or -1 when there is
  // nothing to read.
  auto issue = [&](int stage, int id) -> int {
    if (!kv8_page_ok(g, id)) {
      if (id != -2 && lane == 0) atomicCAS(p.err, 0, kDevErrIndex);
      return -1;
    }
    const int t = prod.unit * kDecUnit + warp * 16;
    const int eoff = id * g.Hkv + prod.seg;  // (the host bounds num_pages * Hkv)
    const long long off = (long long)eoff * (g.page * D) + (t & (g.page - 1)) * D;
    const uint8_t *ks = p.k + off + lane * 16, *vs = p.v + off + lane * 16;
    const uint32_t dk = ring + stage * C::kStageBytes;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      // (D = 128: rows 4 i .., so the exchanged piece alternates)
      const uint32_t d = D == 128 && (i & 1) ? (dk ^ 64) + i * 512 : dk + i * 512;
      cp_async16(d, ks + i * 512);
      cp_async16(d + 16 * D, vs + i * 512);
    }
    return eoff;
  };

  // Exponents are loaded one step before their use, a step after their page
  // is known: nothing waits for them.
  int eo[kStages - 1];
  int next_id = fetch_page();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    eo[s] = -1;
    if (s < nsteps) {
      eo[s] = issue(s, next_id);
      dec_advance(p, prod, segs);
      next_id = s + 1 < nsteps ? fetch_page() : -2;
    }
    cp_async_commit();
  }
  int eo_now = eo[0];
  int ke_now = eo_now >= 0 ? p.ke[eo_now] : 0, ve_now = eo_now >= 0 ? p.ve[eo_now] : 0;

  int step = 0, seg_index = 0, stage = 0;
  while (step < nsteps) {
    // ---------------------------------------------------------- one segment
    const int b = cons.b, h = cons.seg;
    const int len = cons.len;
    const int n_here = min(cons.units - cons.unit, nsteps - step);
    const bool whole = cons.unit == 0 && n_here == cons.units;
    bool bad = false;
    const int rows = seq_rows(p, b, &bad);
    const int r_end = rows * p.G;
    const int vis_min = rows > 0 ? row_sees(p, 0, len, rows) : len;  // the first query's
    // Queries as the 8-wide operand: this lane holds parts of rows 8 t + q8,
    // and the statistics of rows 8 t + 2 c4 and 8 t + 2 c4 + 1.
    float f[C::kQShared ? 1 : kNT][2] = {};
    uint32_t qf[C::kQShared ? 1 : kNT][kSteps][2];
    if constexpr (C::kQShared) __syncthreads();  // the last segment's are read
#pragma unroll
    for (int t0 = 0; t0 < kNT; t0 += C::kQShared ? kDecWarps : 1) {
      const int t = C::kQShared ? t0 + warp : t0;  // (shared: a warp a tile)
      if (C::kQShared && t >= kNT) break;
      const int r = 8 * t + q8;
      const bool on = r < r_end;
      const int i = row_query(p, r);
      const __nv_bfloat16 *src =
          p.q + (((long long)b * p.H + h * p.G + (r - i * p.G)) * p.Nq + i) * D + c4 * kChunks * 16;
      uint2 w[kSteps];
      uint32_t am = 0;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        w[ks] = on ? *reinterpret_cast<const uint2 *>(src + 4 * ks) : make_uint2(0, 0);
        am = max_u16x2(am, w[ks].x & 0x7fff7fffu);
        am = max_u16x2(am, w[ks].y & 0x7fff7fffu);
      }
      am = max(am & 0xffffu, am >> 16);
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      int ea = (int)(am >> 7) - 127;
      if (am < 0x80u || am >= 0x7f80u) ea = 0;  // no normal value, or not finite
      ea = min(ea, 126);
      const float sc = exp2i(-ea);
      const float fr = p.scale_log2 * exp2i(ea);
      if constexpr (C::kQShared) {
#pragma unroll
        for (int ks = 0; ks < kSteps; ks += 2)
          q_ops[(t * (kSteps / 2) + ks / 2) * 32 + lane] =
              make_uint4(bf16x2_to_f16x2_scaled(w[ks].x, sc), bf16x2_to_f16x2_scaled(w[ks].y, sc),
                         bf16x2_to_f16x2_scaled(w[ks + 1].x, sc),
                         bf16x2_to_f16x2_scaled(w[ks + 1].y, sc));
        if (c4 == 0) q_fac[r] = fr;
      } else {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
          qf[t][ks][0] = bf16x2_to_f16x2_scaled(w[ks].x, sc);
          qf[t][ks][1] = bf16x2_to_f16x2_scaled(w[ks].y, sc);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) f[t][x] = __shfl_sync(0xffffffffu, fr, (2 * c4 + x) * 4);
      }
    }
    if constexpr (C::kQShared) __syncthreads();
    // factors of this lane's two rows of a tile, and the positions a row sees
    auto factors = [&](int t) -> uint64_t {
      if constexpr (C::kQShared)
        return *reinterpret_cast<const uint64_t *>(q_fac + 8 * t + 2 * c4);
      const int i = C::kQShared ? 0 : t;
      return f2_pack(f[i][0], f[i][1]);
    };
    auto sees = [&](int t, int x) -> int {
      const int r = 8 * t + 2 * c4 + x;
      return r < r_end ? row_sees(p, row_query(p, r), len, rows) : 0;
    };

    float o[kNT][kSteps][4];
    float nm[kNT][2], dm[kNT][2], l[kNT][2];  // -m; m - M + lift; l
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
#pragma unroll
      for (int j = 0; j < kSteps; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.f;
      nm[t][0] = nm[t][1] = -kDecNone;
      dm[t][0] = dm[t][1] = kDecNoLift;
      l[t][0] = l[t][1] = 0.f;
    }

#pragma unroll 1
    for (int n = 0; n < n_here; ++n, ++step) {
      // issue the step kStages - 1 ahead, then wait for this one's copies
      const bool none = eo_now < 0;
      const float fk = exp2i(max(ke_now, -126)), ev = (float)ve_now;
      eo_now = eo[1];
      int eo_new = -1;
      const int ahead = stage == 0 ? kStages - 1 : stage - 1;
      if (step + kStages - 1 < nsteps) {
        eo_new = issue(ahead, next_id);
        dec_advance(p, prod, segs);
        next_id = step + kStages < nsteps ? fetch_page() : -2;
      }
      cp_async_commit();
#pragma unroll
      for (int i = 0; i + 1 < kStages - 1; ++i) eo[i] = eo[i + 1];
      eo[kStages - 2] = eo_new;
      ke_now = eo_now >= 0 ? p.ke[eo_now] : 0;
      ve_now = eo_now >= 0 ? p.ve[eo_now] : 0;
      cp_async_wait<kStages - 1>();
      __syncwarp();  // every lane's copies of this step
      const uint8_t *st = smem + (warp * kStages + stage) * C::kStageBytes;
      stage = stage == kStages - 1 ? 0 : stage + 1;
      const int t0 = (cons.unit + n) * kDecUnit + warp * 16;
      if (none) continue;  // no positions of this warp (warp-uniform)

      // S^T = K Q^T: 16 positions x 8 rows a tile; s[t][0, 1]: position q8,
      // rows 2 c4 and 2 c4 + 1; s[t][2, 3]: position q8 + 8
      float s[kNT][4];
#pragma unroll
      for (int t = 0; t < kNT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const uint4 w0 = *reinterpret_cast<const uint4 *>(st + (k_get ^ (16 * j)));
        const uint4 w1 = *reinterpret_cast<const uint4 *>(st + (k_get ^ (16 * j)) + 8 * D);
        const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x2x2(x0[i], a0, a2);
          e4m3x4_to_f16x2x2(x1[i], a1, a3);
#pragma unroll
          for (int t = 0; t < kNT; ++t) {
            if constexpr (C::kQShared) {
              const uint2 qv = reinterpret_cast<const uint2 *>(
                  q_ops + (t * (kSteps / 2) + 2 * j + i / 2) * 32 + lane)[i & 1];
              mma_f16(s[t], a0, a1, a2, a3, qv.x, qv.y);
            } else {
              mma_f16(s[t], a0, a1, a2, a3, qf[t][4 * j + i][0], qf[t][4 * j + i][1]);
            }
          }
        }
      }
      const bool edge = t0 + 16 > vis_min;
      // z = s - m (log2 units); while no score passes m by more than 2^tau and
      // no m + ve passes M, the references stay and nothing has to be reduced
      // across the warp.  (Two rows an instruction where there is one.)
      const uint64_t fk2 = f2_pack(fk, fk), ev2 = f2_pack(ev, ev);
      float z[kNT][4];
      float top = -INFINITY, most = -INFINITY;
#pragma unroll
      for (int t = 0; t < kNT; ++t) {
        const uint64_t fx = f2_mul(factors(t), fk2), nm2 = f2_pack(nm[t][0], nm[t][1]);
        f2_unpack(f2_fma(f2_pack(s[t][0], s[t][1]), fx, nm2), z[t][0], z[t][1]);
        f2_unpack(f2_fma(f2_pack(s[t][2], s[t][3]), fx, nm2), z[t][2], z[t][3]);
        if (edge) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int see = sees(t, x);
            if (t0 + q8 >= see) z[t][x] = -INFINITY;
            if (t0 + q8 + 8 >= see) z[t][2 + x] = -INFINITY;
          }
        }
        top = max3(max3(top, z[t][0], z[t][1]), z[t][2], z[t][3]);
        float d0, d1;
        f2_unpack(f2_add(f2_pack(dm[t][0], dm[t][1]), ev2), d0, d1);
        most = max3(most, d0, d1);
      }
      if (__any_sync(0xffffffffu, top > kDecTau || most > kDecLift)) {
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
          float fx[2];
          f2_unpack(f2_mul(factors(t), fk2), fx[0], fx[1]);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const bool see0 = z[t][x] != -INFINITY, see1 = z[t][2 + x] != -INFINITY;
            const float m = -nm[t][x];
            float mx = fmaxf(see0 ? s[t][x] * fx[x] : -INFINITY,
                             see1 ? s[t][2 + x] * fx[x] : -INFINITY);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float m_new = mx > m + kDecTau ? mx : m;
            l[t][x] *= ex2_approx(m - m_new);
            nm[t][x] = -m_new;
            if (see0) z[t][x] = fmaf(s[t][x], fx[x], -m_new);
            if (see1) z[t][2 + x] = fmaf(s[t][2 + x], fx[x], -m_new);
            // M = m - dm + lift: the larger of itself and m + ve
            const float kept = dm[t][x] + (m_new - m);
            const float d_new = fminf(kept, kDecLift - ev);
            const float up = ex2_approx(d_new - kept);
            dm[t][x] = d_new;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              o[t][j][x] *= up;
              o[t][j][2 + x] *= up;
            }
          }
        }
      }
      uint32_t pb[kNT][2];
#pragma unroll
      for (int t = 0; t < kNT; ++t) {
        // P = 2^(s - m), P' = P 2^(m + ve - M + lift)
        float d[2], e[4], pr[4];
        f2_unpack(f2_add(f2_pack(dm[t][0], dm[t][1]), ev2), d[0], d[1]);
#pragma unroll
        for (int x = 0; x < 4; ++x) e[x] = ex2_approx(z[t][x]);
        const uint64_t lift = f2_pack(ex2_approx(d[0]), ex2_approx(d[1]));
        const uint64_t e01 = f2_pack(e[0], e[1]), e23 = f2_pack(e[2], e[3]);
        f2_unpack(f2_add(f2_pack(l[t][0], l[t][1]), f2_add(e01, e23)), l[t][0], l[t][1]);
        f2_unpack(f2_mul(e01, lift), pr[0], pr[1]);
        f2_unpack(f2_mul(e23, lift), pr[2], pr[3]);
        // as the 8-wide operand: positions 2 c4, 2 c4 + 1 (and + 8) of row q8
        pb[t][0] = transpose8x8(pack_f16x2(pr[0], pr[1]));
        pb[t][1] = transpose8x8(pack_f16x2(pr[2], pr[3]));
      }
      // O^T += V^T P'^T: lane q8's columns of tile j are kRun q8 + 2 j, + 1
      uint32_t w[4][kVw];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // positions 2 c4, 2 c4 + 1, and these + 8
        const uint8_t *sv = st + 16 * D + v_get[i & 1] + (i >> 1) * 8 * D;
        if constexpr (D == 128) {
          const uint4 y = *reinterpret_cast<const uint4 *>(sv);
          w[i][0] = y.x;
          w[i][1] = y.y;
          w[i][2] = y.z;
          w[i][3] = y.w;
        } else {
          const uint2 y = *reinterpret_cast<const uint2 *>(sv);
          w[i][0] = y.x;
          w[i][1] = y.y;
        }
      }
      __syncwarp();  // this step's slot is read: the next copies may take it
      bool by_query = false;
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
        by_query = __any_sync(0xffffffffu, odd);
      }
      if (!by_query) {
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          const uint32_t sel = j & 1 ? 0x7362 : 0x5140;
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x2x2(__byte_perm(w[0][j >> 1], w[1][j >> 1], sel), a0, a1);
          e4m3x4_to_f16x2x2(__byte_perm(w[2][j >> 1], w[3][j >> 1], sel), a2, a3);
#pragma unroll
          for (int t = 0; t < kNT; ++t) mma_f16(o[t][j], a0, a1, a2, a3, pb[t][0], pb[t][1]);
        }
      } else {
        // a NaN that some rows see and others do not: query by query, without
        // the positions that one does not see
#pragma unroll 1
        for (int i = 0; i < rows; ++i) {
          const int see = row_sees(p, i, len, rows);
          uint32_t v[4][kVw];
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int y = 0; y < kVw; ++y)
              v[k][y] = t0 + 2 * c4 + (k & 1) + (k >> 1) * 8 < see ? w[k][y] : 0u;
#pragma unroll
          for (int t = 0; t < kNT; ++t) {
            const int ra = 8 * t + 2 * c4;
            const bool on0 = row_query(p, ra) == i, on1 = row_query(p, ra + 1) == i;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              const uint32_t sel = j & 1 ? 0x7362 : 0x5140;
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16x2x2(__byte_perm(v[0][j >> 1], v[1][j >> 1], sel), a0, a1);
              e4m3x4_to_f16x2x2(__byte_perm(v[2][j >> 1], v[3][j >> 1], sel), a2, a3);
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(d, a0, a1, a2, a3, pb[t][0], pb[t][1]);
              if (on0) {
                o[t][j][0] += d[0];
                o[t][j][2] += d[2];
              }
              if (on1) {
                o[t][j][1] += d[1];
                o[t][j][3] += d[3];
              }
            }
          }
        }
      }
    }

    // ---------------------------------------------------------- join the warps
    // kJoin tiles of eight rows at a time.  (One at a time, with two barriers and
    // its own copy of the code each: 37.0 -> 35.0 us for 40 rows of 16 sequences.)
#pragma unroll
    for (int tj = 0; tj < kNT; tj += C::kJoin) {
      if (8 * tj >= r_end) break;
      __syncthreads();  // the merge buffer is free
#pragma unroll
      for (int t = tj; t < kNT && t < tj + C::kJoin; ++t) {
        if (8 * t >= r_end) break;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float ls = l[t][x];
          ls += __shfl_xor_sync(0xffffffffu, ls, 4);
          ls += __shfl_xor_sync(0xffffffffu, ls, 8);
          ls += __shfl_xor_sync(0xffffffffu, ls, 16);
          const int row = warp * C::kMergeRows + 8 * (t - tj) + 2 * c4 + x;
          if (q8 == 0)
            *reinterpret_cast<float4 *>(merge_s + row * 4) =
                make_float4(-nm[t][x], kDecLift - dm[t][x] - nm[t][x], ls, 0.f);
          float *d = merge_o + row * C::kRowStride + q8 * C::kRunStride;
#pragma unroll
          for (int j = 0; j < kSteps; j += 2)
            *reinterpret_cast<float4 *>(d + 2 * j) = make_float4(
                o[t][j][x], o[t][j][2 + x], o[t][j + 1][x], o[t][j + 1][2 + x]);
        }
      }
      __syncthreads();
      constexpr int kPer = kDecThreads / 8;  // threads of a row
      constexpr int kCols = D / kPer;        // columns of a thread
      const int col = (threadIdx.x % kPer) * kCols;
#pragma unroll 1
      for (int t = tj; t < kNT && t < tj + C::kJoin; ++t) {
        const int row = 8 * (t - tj) + threadIdx.x / kPer;
        const int r = 8 * tj + row;
        if (r >= r_end) break;
        float mm = kDecNone, mmo = kDecNone, ll = 0.f;
        float4 st[kDecWarps];
#pragma unroll
        for (int w2 = 0; w2 < kDecWarps; ++w2) {
          st[w2] = *reinterpret_cast<const float4 *>(merge_s + (w2 * C::kMergeRows + row) * 4);
          mm = fmaxf(mm, st[w2].x);
          mmo = fmaxf(mmo, st[w2].y);
        }
        float out[kCols];
#pragma unroll
        for (int j = 0; j < kCols; ++j) out[j] = 0.f;
        const float *d0 = merge_o + row * C::kRowStride + (col / C::kRun) * C::kRunStride +
                          col % C::kRun;
#pragma unroll
        for (int w2 = 0; w2 < kDecWarps; ++w2) {
          // nothing seen: l is 0 (a NaN score leaves l NaN, which has to stay)
          const bool none = st[w2].z == 0.f;
          ll += none ? 0.f : st[w2].z * ex2_approx(st[w2].x - mm);
          const float wt = none ? 0.f : ex2_approx(st[w2].y - mmo);
          const float *d = d0 + w2 * C::kMergeRows * C::kRowStride;
#pragma unroll
          for (int j = 0; j < kCols; j += 4) {
            const float4 y = *reinterpret_cast<const float4 *>(d + j);
            out[j] = fmaf(wt, y.x, out[j]);
            out[j + 1] = fmaf(wt, y.y, out[j + 1]);
            out[j + 2] = fmaf(wt, y.z, out[j + 2]);
            out[j + 3] = fmaf(wt, y.w, out[j + 3]);
          }
        }
        if (whole) {
          const int i = row_query(p, r);
          const long long orow = ((long long)b * p.H + h * p.G + (r - i * p.G)) * p.Nq + i;
          // 2^(M - lift - m) / l, in two factors (M - m is a value exponent)
          const float half = ll == 0.f ? 0.f : ex2_approx(0.5f * (mmo - kDecLift - mm));
          const float inv = ll == 0.f ? 0.f : half / ll;
          uint2 *dst = reinterpret_cast<uint2 *>(p.o + orow * D + col);
#pragma unroll
          for (int j = 0; j < kCols; j += 4)
            dst[j / 4] = make_uint2(pack_bf16x2(out[j] * inv * half, out[j + 1] * inv * half),
                                    pack_bf16x2(out[j + 2] * inv * half, out[j + 3] * inv * half));
          if (col == 0)
            p.lse[orow] =
                ll == 0.f ? -INFINITY : (mm + lg2_approx(ll)) * 0.69314718055994531f;
        } else {
          float *d = p.part + (((size_t)blockIdx.x * 2 + (seg_index > 0)) * C::kRows + r) *
                                  (D + 4);
#pragma unroll
          for (int j = 0; j < kCols; j += 4)
            *reinterpret_cast<float4 *>(d + col + j) =
                make_float4(out[j], out[j + 1], out[j + 2], out[j + 3]);
          if (col == 0) *reinterpret_cast<float4 *>(d + D) = make_float4(mm, mmo, ll, 0.f);
        }
      }
    }
    // next segment
    ++seg_index;
    cons.unit += n_here - 1;
    dec_advance(p, cons, segs);
  }
}

// One row's n partials joined by a block: a warp takes every eighth, its lanes
// D/32 columns each; then the warps.  at(i): partial i, O relative to 2^M with
// m, M and l behind it.
constexpr int kMergeWarps = 8;
template <int D, typename At>
__device__ __forceinline__ void merge_row(At at, int n, __nv_bfloat16 *o, float *lse) {
  constexpr int kPer = D / 32;
  __shared__ float stat[kMergeWarps][3];
  __shared__ float cols[kMergeWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float mm = kDecNone, mmo = kDecNone, ll = 0.f, acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
  constexpr int kDeep = 4;  // partials in flight
#pragma unroll 1
  for (int c = warp; c < n; c += kMergeWarps * kDeep) {
    float4 st[kDeep];
    float x[kDeep][kPer];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int ci = c + i * kMergeWarps;
      st[i] = make_float4(kDecNone, kDecNone, 0.f, 0.f);
      if (ci < n) {
        const float *d = at(ci);
        st[i] = *reinterpret_cast<const float4 *>(d + D);
#pragma unroll
        for (int k = 0; k < kPer; ++k) x[i][k] = d[lane * kPer + k];
      }
    }
    float m_new = mm, mo_new = mmo;
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      m_new = fmaxf(m_new, st[i].x);
      mo_new = fmaxf(mo_new, st[i].y);
    }
    ll *= ex2_approx(mm - m_new);
    const float up = ex2_approx(mmo - mo_new);
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] *= up;
    mm = m_new;
    mmo = mo_new;
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      // nothing seen: l is 0 (a NaN score leaves l NaN, which has to stay)
      if (st[i].z == 0.f) continue;
      ll += st[i].z * ex2_approx(st[i].x - mm);
      const float wt = ex2_approx(st[i].y - mmo);
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(wt, x[i][k], acc[k]);
    }
  }
  if (lane == 0) {
    stat[warp][0] = mm;
    stat[warp][1] = mmo;
    stat[warp][2] = ll;
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) cols[warp][lane * kPer + k] = acc[k];
  __syncthreads();
  if (threadIdx.x >= D) return;
  mm = mmo = kDecNone;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    mm = fmaxf(mm, stat[w][0]);
    mmo = fmaxf(mmo, stat[w][1]);
  }
  ll = 0.f;
  float out = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    if (stat[w][2] == 0.f) continue;
    ll += stat[w][2] * ex2_approx(stat[w][0] - mm);
    out = fmaf(ex2_approx(stat[w][1] - mmo), cols[w][threadIdx.x], out);
  }
  const float half = ll == 0.f ? 0.f : ex2_approx(0.5f * (mmo - kDecLift - mm));
  const float inv = ll == 0.f ? 0.f : half / ll;
  o[threadIdx.x] = __float2bfloat16(out * inv * half);
  if (threadIdx.x == 0)
    *lse = ll == 0.f ? -INFINITY : (mm + lg2_approx(ll)) * 0.69314718055994531f;
}

// The same by a warp, for rows of few partials.
template <int D, typename At>
__device__ __forceinline__ void merge_row_warp(At at, int n, __nv_bfloat16 *o, float *lse) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  float mm = kDecNone, mmo = kDecNone, ll = 0.f, acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
  constexpr int kDeep = 8;  // partials in flight
#pragma unroll 1
  for (int c = 0; c < n; c += kDeep) {
    float4 st[kDeep];
    float x[kDeep][kPer];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      st[i] = make_float4(kDecNone, kDecNone, 0.f, 0.f);
      if (c + i < n) {
        const float *d = at(c + i);
        st[i] = *reinterpret_cast<const float4 *>(d + D);
#pragma unroll
        for (int k = 0; k < kPer; ++k) x[i][k] = d[lane * kPer + k];
      }
    }
    float m_new = mm, mo_new = mmo;
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      m_new = fmaxf(m_new, st[i].x);
      mo_new = fmaxf(mo_new, st[i].y);
    }
    ll *= ex2_approx(mm - m_new);
    const float up = ex2_approx(mmo - mo_new);
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] *= up;
    mm = m_new;
    mmo = mo_new;
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      if (st[i].z == 0.f) continue;  // nothing seen
      ll += st[i].z * ex2_approx(st[i].x - mm);
      const float wt = ex2_approx(st[i].y - mmo);
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(wt, x[i][k], acc[k]);
    }
  }
  const float half = ll == 0.f ? 0.f : ex2_approx(0.5f * (mmo - kDecLift - mm));
  const float inv = ll == 0.f ? 0.f : half / ll;
  uint32_t *dst = reinterpret_cast<uint32_t *>(o + lane * kPer);
#pragma unroll
  for (int k = 0; k < kPer / 2; ++k)
    dst[k] = pack_bf16x2(acc[2 * k] * inv * half, acc[2 * k + 1] * inv * half);
  if (lane == 0) *lse = ll == 0.f ? -INFINITY : (mm + lg2_approx(ll)) * 0.69314718055994531f;
}

// Merge of the runs' partial results; segments that one run held whole are
// already written.  A block a row, or (kWarpRow) a warp: with many rows each has
// few partials, and a block's common part is paid for eight rows.
template <int D, bool kWarpRow>
__global__ void __launch_bounds__(kMergeWarps * 32)
    tk_kv8_merge_kernel(const __grid_constant__ Kv8AttnParams p) {
  __shared__ int red[2][kMergeWarps];
  // (It does not let its dependents begin: the next call's runs, resident early,
  // would take the registers that these blocks need; 161 -> 228 us at 8 x 16384.)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x, b = blockIdx.y;
  const int r = kWarpRow ? blockIdx.z * kMergeWarps + warp : blockIdx.z;
  bool bad = false;
  const int rows = seq_rows(p, b, &bad);
  // the units before this sequence, and all of them
  int before = 0, total = 0;
#pragma unroll 1
  for (int x = threadIdx.x; x < p.B; x += kMergeWarps * 32) {
    const int v = seq_units(p, x, kDecUnit) * p.g.Hkv;
    total += v;
    if (x < b) before += v;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  if (lane == 0) {
    red[0][warp] = before;
    red[1][warp] = total;
  }
  __syncthreads();
  before = total = 0;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    before += red[0][w];
    total += red[1][w];
  }
  const int units = seq_units(p, b, kDecUnit);
  const int share = max(1, (int)(((unsigned)total + p.ctas - 1) / (unsigned)p.ctas));
  const int s0 = before + h * units;
  const int c0 = s0 / share, c1 = (s0 + max(units, 1) - 1) / share;
  // run c0's partial is its first segment's only if it starts where the segment does
  const int first0 = c0 * share == s0 ? 0 : 1;
  const float *base = p.part + (size_t)r * (D + 4);
  const size_t slot = (size_t)p.tile_rows * (D + 4);
  // All above reads only what the launch before leaves alone, and what came
  // before that one has ended (it starts this one after its own wait).
  grid_wait();
  if (r >= rows * p.G || c0 == c1) return;
  const int i = row_query(p, r);
  const long long orow = ((long long)b * p.H + h * p.G + (r - i * p.G)) * p.Nq + i;
  const auto at = [&](int k) {
    return base + ((size_t)(c0 + k) * 2 + (k == 0 ? first0 : 0)) * slot;
  };
  if constexpr (kWarpRow)
    merge_row_warp<D>(at, c1 - c0 + 1, p.o + orow * D, p.lse + orow);
  else
    merge_row<D>(at, c1 - c0 + 1, p.o + orow * D, p.lse + orow);
}

}  // namespace tkattn
