// tk_kv8_chunk.cuh -- attention of many query rows over the 8-bit paged cache
// (prefill chunks, many drafted tokens, wide head groups) on the tensor cores.
//
// The operation is tk_kv8_decode.cuh's; here a (sequence, key/value head) has
// more query rows than that kernel's tiles.  Rows r = i * G + g are cut into
// units of 256 (two tiles of 128); a unit visits the 128-position key tiles
// its rows see.  The list of (unit, key tile) steps is cut into equal runs, one
// for each CTA (the lengths live on the device, every CTA finds its run); a unit
// that several runs share leaves partial results that a second kernel merges.
//
// Products:
//   S = Q K^T   kind::f8f6f4: the key codes go to the tensor core as they lie
//               in the cache.  A query row is scaled by a power of two to a
//               largest magnitude in [128, 256) and split in two E4M3 terms,
//               hi = rn(q), lo = rn(q - hi): bf16's eight bits are two times
//               E4M3's four, so the split is exact but for elements below 2^-9
//               of the row's largest (off by at most 2^-17 of it).  Two fp8
//               products take the time of one in bf16 and no conversion.
//               Each page's 2^ke multiplies its scores in fp32.
//   O = P V     kind::f16: P in fp16 (four times bf16's precision), the value
//               codes converted to fp16 in shared memory and multiplied by
//               2^(ve - E + 6), E the largest value exponent of the run so far
//               (exact while a page's lies within 2^21 of it); when E grows, O
//               is rescaled.
// The softmax is tk_attn_fwd.cuh's: one thread a row, a lazily moved maximum,
// the fp32 sum of the unrounded P, the rounding of each tile's largest P
// carried into the divisor.
//
// With at most 128 rows a (sequence, head) at D = 64 (kPair) both tiles hold the same rows
// and take every other key tile: a step is two key tiles, the tiles' results are
// joined at the end (or both left as partials), and the softmax of one works beside the other's
// products as it does with 256 rows.
//
// Roles (one CTA an SM, 512 threads):
//   warps 0-3, 4-7  softmax of tile 0, 1; at a unit's start they convert their
//                   tile's queries (their last scores being in hand, no product
//                   still reads them)
//   warps 8-11      value conversion, and the epilogue
//   warp 12         tensor-core issue
//   warps 13, 14    TMA loads of values and of keys, a lane a page
//   warp 15         the run's segments, which the other roles read
// A NaN value code would spread over a tile's rows through 0 * NaN: codes are
// replaced by 0 and the first position of each column that held one is kept;
// rows that see that position get NaN in that column.
//
// Bound by the tensor core and, almost as much, by the softmax and value
// conversion beside it: 2048 queries behind 14336 positions of 32 heads of 128 over 8 key
// heads take 433 us, 1190 TFLOP/s, 62 % of a cuBLAS product's rate (this library's
// dense forward pass over bf16 reaches 1330 unmasked).  A step of two tiles takes some 4000
// cycles of which the products are 2048; instruction fetch counts: one loader
// warp, roles that each post their own segments and unrolled loops took 780 us.
//
// Every wait is bounded as in tk_attn_fwd.cuh.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "sm103_ptx.cuh"
#include "tk_device.h"
#include "tk_kv8.h"
#include "tk_kv8_copy.cuh"
#include "tk_kv8_decode.cuh"

namespace tkattn {

constexpr int kChunkThreads = 512;
constexpr int kChunkRows = 256;   // query rows of a unit
constexpr float kChunkTau = 8.f;  // lazy maximum: P <= 2^8
constexpr int kChunkLift = 6;     // value codes are lifted by 2^6

template <int D>
struct ChunkCfg {
  static constexpr int kRaw = 128 * D;                   // a tile of codes
  static constexpr int kQTile = D == 128 ? 32768 : 16384;  // hi and lo of 128 rows
  static constexpr int kKs = D == 128 ? 3 : 4;           // key ring
  static constexpr int kVs = D == 128 ? 2 : 4;           // value ring
  static constexpr int kV16 = 128 * D * 2;               // a converted value tile
  static constexpr int kV16s = 2;  // (the issue loop flips between them)
  static constexpr int kOffK = 2 * kQTile;
  static constexpr int kOffV = kOffK + kKs * kRaw;
  static constexpr int kOffV16 = kOffV + kVs * kRaw;
  static constexpr int kSmem = kOffV16 + kV16s * kV16;
  static constexpr int kSmemAlloc = kSmem + 1024;  // + alignment slack
  static constexpr uint32_t kColS0 = 0, kColS1 = 128, kColO0 = 256, kColO1 = 256 + D;
};

// A segment: the part of one unit that lies in a CTA's run.
struct ChunkSeg {
  int b, h, mb;     // mb < 0: the run is over
  int j0, n;        // its steps
  int n0, n1;       // how many of them each tile of queries takes part in
  int len, rows;    // of the sequence
  int whole;        // the unit lies in this run alone
};

struct ChunkShared {
  uint64_t q_full[2];     // tile's queries converted        (4 softmax warps)
  uint64_t k_full[4];     // key tile landed                 (1 + tx)
  uint64_t k_empty[4];    // both tiles' S done with it      (commit)
  uint64_t v_full[4];     // value tile landed               (1 + tx)
  uint64_t v_empty[4];    // converted                       (4 converter warps)
  uint64_t v_ready[2];    // fp16 values ready               (4 converter warps)
  uint64_t v_free[2];     // both tiles' P V done with them  (commit)
  uint64_t s_full[2];     // S of tile t complete            (commit)
  uint64_t p_full[2];     // P of tile t written             (4 softmax warps)
  uint64_t fin_full[2][2];  // [parity][tile] final m, l     (4 softmax warps)
  uint64_t o_full[2];     // tile's last P V of a unit done  (commit)
  uint64_t o_free[2];     // epilogue has read O             (4 converter warps)
  uint64_t conv_bar;      // converter warps, once a unit    (4 converter warps)
  uint64_t seg_full[4];   // segment posted                  (1)
  uint64_t seg_empty[4];  // every role has read it          (15: 8 + 4 warps, issue, 2 loads)
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  // run
  Kv8Place place;
  long long red[kChunkThreads / 32];
  ChunkSeg seg[4];
  // per step, eight deep: a slot is rewritten only when every reader is four steps on
  alignas(16) float k_scale[8][8];  // 2^ke of the tile's eight runs of 16 positions
  int k_valid[8];         // bit g: run g lies in a page that could be read
  int v_exp8[8][8];       // value exponents of the runs
  int v_valid[8];         // as k_valid, for the values
  int v_exp[2];           // exponent the converted tile carries (6 - E)
  float m_fin[2][2][128], l_fin[2][2][128], lc_fin[2][2][128];  // [parity][tile][row]
  // eight segments deep: a converter warp is at most two tiles ahead of another
  int nan_any[8];
  int nan_pos[8][128];    // [segment][column]: first position that held a NaN
};

__device__ __forceinline__ void chunk_abort(ChunkShared &sb, int *err) {
  sb.abort = 1;
  atomicCAS(err, 0, kDevErrTimeout);
}

// Key tiles that rows [first, first + 128) of a sequence with `rows` queries
// and length len visit (0: no such row).
__device__ __forceinline__ int chunk_tiles(const Kv8AttnParams &p, int first, int len, int rows) {
  const int r_end = rows * p.G;
  if (first >= r_end) return 0;
  const int i = row_query(p, min(first + 127, r_end - 1));
  return max(1, (row_sees(p, i, len, rows) + 127) / 128);
}

struct ChunkSeq {
  int len, rows, units;  // units: 256-row units of a head
};
__device__ __forceinline__ ChunkSeq chunk_seq(const Kv8AttnParams &p, int b) {
  bool bad = false;
  ChunkSeq s;
  s.len = seq_len(p, b, &bad);
  s.rows = seq_rows(p, b, &bad);
  s.units = (s.rows * p.G + kChunkRows - 1) / kChunkRows;
  return s;
}
// Steps of unit mb: the key tiles of its last row, or pairs of them.
__device__ __forceinline__ int chunk_cost(const Kv8AttnParams &p, const ChunkSeq &s, int mb) {
  const int last = min(mb * kChunkRows + kChunkRows, s.rows * p.G) - 1;
  const int tiles = max(1, (row_sees(p, row_query(p, last), s.len, s.rows) + 127) / 128);
  return p.pair ? (tiles + 1) / 2 : tiles;
}
// A head's units together: by one thread, or by a warp.
__device__ __forceinline__ long long chunk_seq_cost(const Kv8AttnParams &p, int b) {
  const ChunkSeq s = chunk_seq(p, b);
  long long c = 0;
#pragma unroll 1
  for (int mb = 0; mb < s.units; ++mb) c += chunk_cost(p, s, mb);
  return c;
}
__device__ __forceinline__ long long chunk_seq_cost_warp(const Kv8AttnParams &p, int b, int lane) {
  const ChunkSeq s = chunk_seq(p, b);
  long long c = 0;
#pragma unroll 1
  for (int mb = lane; mb < s.units; mb += 32) c += chunk_cost(p, s, mb);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) c += __shfl_xor_sync(0xffffffffu, c, d);
  return c;
}

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, uint64_t *bar,
                                            int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y)
      : "memory");
}

// D[tmem] (+)= A[smem] B[smem]^T, E4M3 operands, fp32 accumulation.
template <uint32_t kAcc>
__device__ __forceinline__ void umma_f8_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi,
                                           uint32_t b_lo, uint32_t b_hi, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(kAcc)
      : "memory");
}

// kind::f8f6f4, E4M3 x E4M3 -> fp32, both operands K-major (format codes 0).
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// High word of a descriptor with the 64-byte swizzle.
__host__ __device__ constexpr uint32_t sdesc_sw64_hi(uint32_t sbo) {
  return ((sbo >> 4) & 0x3FFFu) | (1u << 14) | (4u << 29);
}

// Convert one tile's query rows: warp w of the tile takes rows [32 w, 32 w + 32).
// Returns this lane's row's score factor scale_log2 * 2^(its exponent).
template <int D>
__device__ __forceinline__ float chunk_queries(const Kv8AttnParams &p, int b, int h, int first,
                                               int r_end, int w, int lane, uint8_t *tile) {
  constexpr int kLanes = D / 8;           // lanes of a row, 8 values each
  constexpr int kPerIt = 32 / kLanes;     // rows a pass
  constexpr int kIts = 32 / kPerIt;
  constexpr int kDeep = 4;                // passes loaded together, one batch ahead
  const int l = lane % kLanes, sub = lane / kLanes;
  float mine = 1.f;
  auto load = [&](int it) -> uint4 {
    const int r = first + w * 32 + it * kPerIt + sub;
    if (r >= r_end) return make_uint4(0, 0, 0, 0);
    const int i = row_query(p, r);
    return *reinterpret_cast<const uint4 *>(
        p.q + (((long long)b * p.H + h * p.G + (r - i * p.G)) * p.Nq + i) * D + l * 8);
  };
  uint4 ahead[kDeep];
#pragma unroll
  for (int u = 0; u < kDeep; ++u) ahead[u] = load(u);
#pragma unroll 1
  for (int it0 = 0; it0 < kIts; it0 += kDeep) {
    if (first + w * 32 + it0 * kPerIt >= r_end) break;  // no row left (warp-uniform)
    uint4 v[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      v[u] = ahead[u];
      ahead[u] = it0 + kDeep < kIts ? load(it0 + kDeep + u) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int row = w * 32 + (it0 + u) * kPerIt + sub;  // row of the tile
      const uint32_t x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      uint32_t am = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) am = max_u16x2(am, x[i] & 0x7fff7fffu);
      am = max(am & 0xffffu, am >> 16);
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1)
        am = max(am, __shfl_xor_sync(0xffffffffu, am, d));
      int ea = (int)(am >> 7) - 127;
      if (am < 0x80u) ea = 7;  // no normal value
      ea = max(ea, -119);
      const bool odd = am >= 0x7f80u;  // a NaN or an infinity: the row's scores are NaN
      const float sc = odd ? 0.f : exp2i(7 - ea);
      const float fr = odd ? __uint_as_float(0x7fc00000u) : p.scale_log2 * exp2i(ea - 7);
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t hc = 0, lc = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t y = x[2 * i + k];
          const float a = __uint_as_float(y << 16) * sc, c = __uint_as_float(y & 0xffff0000u) * sc;
          const uint32_t code = pack_e4m3x2(a, c);
          const float2 back = e4m3x2_to_float2((uint16_t)code);
          hc |= code << (16 * k);
          lc |= pack_e4m3x2(a - back.x, c - back.y) << (16 * k);
        }
        hi[i] = hc;
        lo[i] = lc;
      }
      const int piece = l >> 1, half = (l & 1) * 8;
      uint8_t *line = tile + row * 128;
      *reinterpret_cast<uint2 *>(line + ((piece ^ (row & 7)) << 4) + half) =
          make_uint2(hi[0], hi[1]);
      if constexpr (D == 128)
        *reinterpret_cast<uint2 *>(line + 16384 + ((piece ^ (row & 7)) << 4) + half) =
            make_uint2(lo[0], lo[1]);
      else
        *reinterpret_cast<uint2 *>(line + (((4 + piece) ^ (row & 7)) << 4) + half) =
            make_uint2(lo[0], lo[1]);
      // lane kPerIt * (it0 + u) + s owns row s of this pass
      const float theirs = __shfl_sync(0xffffffffu, fr, (lane % kPerIt) * kLanes);
      if (lane / kPerIt == it0 + u) mine = theirs;
    }
  }
  return mine;
}

// The x-th segment of the run, as a role reads it; false if the wait was
// abandoned.  Whole warp (or the one thread of a role that has no more).
__device__ __forceinline__ bool chunk_next(ChunkShared &sb, uint32_t x, bool arrive,
                                           volatile int *abort_flag, ChunkSeg &out) {
  if (!mbar_wait(&sb.seg_full[x & 3], (x >> 2) & 1, abort_flag)) return false;
  out = sb.seg[x & 3];
  if (arrive) mbar_arrive(&sb.seg_empty[x & 3]);
  return true;
}

// The loads of the run's key tiles or (kV) value tiles, a lane a page, and what
// the other roles have to know of each: which pages could be read, and their
// factors.  One body for both warps: the code streams of an SM's roles share its
// instruction fetch, which bounds this kernel when they are long.  Page numbers and exponents are fetched 32 pages at a time, one batch
// ahead of their use.
template <int D, bool kPair>
__device__ __forceinline__ void chunk_load(const Kv8AttnParams &p, bool kV, const CUtensorMap *map,
                                           ChunkShared &sb, uint8_t *ring, int lane,
                                           volatile int *abort_flag) {
  using C = ChunkCfg<D>;
  const uint32_t kRing = kV ? C::kVs : C::kKs;
  uint64_t *full = kV ? sb.v_full : sb.k_full, *empty = kV ? sb.v_empty : sb.k_empty;
  const int8_t *exps = kV ? p.ve : p.ke;
  const Kv8Geom &g = p.g;
  const int pages = 128 >> p.page_log2;  // of a tile
  const int batch = 32 / pages;          // tiles of 32 pages
  uint32_t idx = 0;                      // steps loaded
  uint32_t st = 0, turn = 0;             // ring slot of step idx, parity of its use
  bool gone = false;
#pragma unroll 1
  for (uint32_t sx = 0; !gone; ++sx) {
    ChunkSeg sg;
    if (!chunk_next(sb, sx, lane == 0, abort_flag, sg)) {
      if (lane == 0) chunk_abort(sb, p.err);
      break;
    }
    if (sg.mb < 0) break;
    const int first = kPair ? 2 * sg.j0 : sg.j0, n = kPair ? 2 * sg.n : sg.n;  // key tiles
    // lane's page of the batch that starts at tile x of the segment, or -1
    auto fetch = [&](int x) -> int {
      const long long t = (long long)(first + x) * 128 + ((long long)lane << p.page_log2);
      if (x >= n || t >= sg.len || t >= (long long)(first + n) * 128) return -1;
      const int id = p.table[kv8_table_offset(g, sg.b, (int)(t >> p.page_log2))];
      if (kv8_page_ok(g, id)) return id;
      if (!kV) atomicCAS(p.err, 0, kDevErrIndex);
      return -1;
    };
    auto fetch_exp = [&](int id) -> int {
      return id >= 0 ? (int)exps[id * g.Hkv + sg.h] : (kV ? kKv8ExpMin : 0);
    };
    int id = fetch(0), ex = fetch_exp(id);
    int id_next = fetch(batch), ex_next = 0;
#pragma unroll 1
    for (int j = 0; j < n; ++j, ++idx) {
      const int x = j & (batch - 1);  // tile of the batch
      if (x == 0 && j > 0) {
        id = id_next;
        ex = batch > 1 ? ex_next : fetch_exp(id);
        id_next = fetch(j + batch);
      }
      if (x == (batch > 1 ? 1 : 0)) ex_next = fetch_exp(id_next);
      int ok = 1;
      if (lane == 0 && idx >= kRing) ok = mbar_wait(&empty[st], turn ^ 1, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        if (lane == 0) chunk_abort(sb, p.err);
        gone = true;
        break;
      }
      // eight runs of 16 positions, whatever the page
      const int src = x * pages + ((lane & 7) >> (p.page_log2 - 4));
      const int er = __shfl_sync(0xffffffffu, ex, src);
      const int mine = __shfl_sync(0xffffffffu, id, x * pages + (lane & (pages - 1)));
      const uint32_t have = __ballot_sync(0xffffffffu, lane < pages && mine >= 0);
      const uint32_t bits = __ballot_sync(
          0xffffffffu, lane < 8 && (have >> ((lane & 7) >> (p.page_log2 - 4)) & 1));
      if (kV) {
        if (lane < 8) sb.v_exp8[idx & 7][lane] = er;
        if (lane == 0) sb.v_valid[idx & 7] = (int)bits;
      } else {
        if (lane < 8) sb.k_scale[idx & 7][lane] = exp2i(max(er, -126));
        if (lane == 0) sb.k_valid[idx & 7] = (int)bits;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(&full[st], __popc(have) * g.page * D);
      __syncwarp();
      if (lane < pages && mine >= 0)
        tma_load_2d(ring + st * C::kRaw + (lane << p.page_log2) * D, map, &full[st], 0,
                    (mine * g.Hkv + sg.h) << p.page_log2);
      if (++st == kRing) {
        st = 0;
        turn ^= 1;
      }
    }
  }
  // wait for the copies still in flight (all consumed on the normal path)
  if (lane == 0) {
    int never = 0;
#pragma unroll 1
    for (uint32_t s = 0; s < kRing && s < idx; ++s) {
      const uint32_t last = idx - 1 - ((idx - 1 - s) % kRing);
      mbar_wait(&full[s], (last / kRing) & 1, &never);
    }
  }
}

template <int D, bool kPair>
__global__ void __launch_bounds__(kChunkThreads, 1)
    tk_kv8_chunk_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ Kv8AttnParams p) {
  using C = ChunkCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ ChunkShared sb;
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile int *abort_flag = &sb.abort;
  const Kv8Geom &g = p.g;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sb.q_full[t], 4);
      mbar_init(&sb.v_ready[t], 4);
      mbar_init(&sb.v_free[t], 1);
      mbar_init(&sb.s_full[t], 1);
      mbar_init(&sb.p_full[t], 4);
      mbar_init(&sb.fin_full[0][t], 4);
      mbar_init(&sb.fin_full[1][t], 4);
      mbar_init(&sb.o_full[t], 1);
      mbar_init(&sb.o_free[t], 4);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sb.k_full[s], 1);
      mbar_init(&sb.k_empty[s], 1);
      mbar_init(&sb.v_full[s], 1);
      mbar_init(&sb.v_empty[s], 4);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sb.seg_full[s], 1);
      mbar_init(&sb.seg_empty[s], 15);
    }
    mbar_init(&sb.conv_bar, 4);
    mbar_init(&sb.mma_done, 1);
    sb.abort = 0;
    for (int i = 0; i < 8; ++i) sb.nan_any[i] = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < 8 * 128; i += kChunkThreads)
    sb.nan_pos[i >> 7][i & 127] = 0x7fffffff;
  if (warp == 12) {
    tmem_alloc(&sb.tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == 14 && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  grid_wait();
  grid_launch_dependents();  // (after the wait: the merge reads the lengths before its own)
  if (blockIdx.x == 0) {  // report what is out of range, once
    bool bad = false;
#pragma unroll 1
    for (int b = threadIdx.x; b < p.B; b += kChunkThreads) {
      seq_len(p, b, &bad);
      seq_rows(p, b, &bad);
    }
    if (bad) atomicCAS(p.err, 0, kDevErrIndex);
  }
  // The work of each sequence.  Where sequences have many units (the lower
  // bound by the call's sizes) a warp sums one, into shared memory that the
  // rings use later; else, or where those sums would not fit, a thread does.
  long long *sums = reinterpret_cast<long long *>(smem);
  const bool by_warp = p.Nq * p.G > 8 * kChunkRows && p.B <= C::kSmem / 8;
  if (by_warp) {
#pragma unroll 1
    for (int b = warp; b < p.B; b += kChunkThreads / 32) {
      const long long c = chunk_seq_cost_warp(p, b, lane);
      if (lane == 0) sums[b] = c;
    }
    __syncthreads();
  }
  kv8_scan(
      p, [&](int b) { return (by_warp ? sums[b] : chunk_seq_cost(p, b)) * p.g.Hkv; }, blockIdx.x,
      &sb.place, sb.red, blockIdx.x == 0 ? p.prefix : nullptr);
  if (by_warp) fence_proxy_async_smem();  // the sums are read before a copy lands over them
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sb.tmem_base;
  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;\n" ::: "memory");
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;  // row in tile == TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + (t ? C::kColS1 : C::kColS0);
    const uint32_t tO = tmem + lane_off + (t ? C::kColO1 : C::kColO0);
    uint32_t s_phase = 0;
    uint32_t step0 = 0;  // steps of the run before this segment
    uint32_t part = 0;   // segments this tile took part in
#pragma unroll 1
    for (uint32_t x = 0;; ++x) {
      ChunkSeg sg;
      if (!chunk_next(sb, x, lane == 0, abort_flag, sg)) {
        chunk_abort(sb, p.err);
        goto done;
      }
      if (sg.mb < 0) break;
      const int n_t = t ? sg.n1 : sg.n0;
      if (n_t == 0) {
        step0 += sg.n;
        continue;
      }
      const int first = kPair ? 0 : sg.mb * kChunkRows + t * 128;
      const int r_end = sg.rows * p.G;
      const int k_base = sg.j0 * 128, step_end = step0 + sg.n;
      const float c =
          chunk_queries<D>(p, sg.b, sg.h, first, r_end, warp & 3, lane, smem + t * C::kQTile);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb.q_full[t]);
      const int r = first + row;
      const int vis = r < r_end ? row_sees(p, row_query(p, r), sg.len, sg.rows) : 0;
      // Warps whose 32 rows all lie past the last one keep the protocol only.
      const bool idle = first + (warp & 3) * 32 >= r_end;
      const int vis_min = __reduce_min_sync(0xffffffffu, r < r_end ? vis : 0x7fffffff);
      float m_run = -INFINITY, l_run = 0.f, lc_run = 0.f;
      int e_cur = 0;
#pragma unroll 1
      for (int j = 0; j < n_t; ++j) {
        if (!mbar_wait(&sb.s_full[t], s_phase, abort_flag)) {
          chunk_abort(sb, p.err);
          goto done;
        }
        s_phase ^= 1;
        const uint32_t idx = kPair ? 2 * (step0 + j) + t : step0 + j;  // key tiles before
        if (idle) {
          if (!mbar_wait(&sb.v_ready[idx % C::kV16s], (idx / C::kV16s) & 1, abort_flag)) {
            chunk_abort(sb, p.err);
            goto done;
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sb.p_full[t]);
            if (j == n_t - 1) mbar_arrive(&sb.fin_full[part & 1][t]);
          }
          continue;
        }
        tc_fence_after_sync();
        uint32_t s[128];
        tmem_ld_32x32b_x32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
        tmem_ld_32x32b_x32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
        tmem_ld_32x32b_x32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&s[64]));
        tmem_ld_32x32b_x32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&s[96]));
        // each run of 16 positions has its page's factor
        float cg[8];
        {
          const float4 a = *reinterpret_cast<const float4 *>(&sb.k_scale[idx & 7][0]);
          const float4 d = *reinterpret_cast<const float4 *>(&sb.k_scale[idx & 7][4]);
          cg[0] = a.x * c;
          cg[1] = a.y * c;
          cg[2] = a.z * c;
          cg[3] = a.w * c;
          cg[4] = d.x * c;
          cg[5] = d.y * c;
          cg[6] = d.z * c;
          cg[7] = d.w * c;
        }
        const int valid = sb.k_valid[idx & 7];
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 128; ++i) reg_barrier(s[i]);
        const int k0 = kPair ? 2 * (k_base + j * 128) + t * 128 : k_base + j * 128;
        if (k0 + 128 > vis_min || valid != 0xff) {
          const int lim = vis - k0;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int lq = valid >> q & 1 ? lim - 16 * q : 0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i >= lq) s[16 * q + i] = __float_as_uint(-INFINITY);
          }
        }
        float m_cand = -INFINITY;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t *x = &s[16 * q];
          float a = max3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
          float d = max3(__uint_as_float(x[3]), __uint_as_float(x[4]), __uint_as_float(x[5]));
          a = max3(a, __uint_as_float(x[6]), __uint_as_float(x[7]));
          d = max3(d, __uint_as_float(x[8]), __uint_as_float(x[9]));
          a = max3(a, __uint_as_float(x[10]), __uint_as_float(x[11]));
          d = max3(d, __uint_as_float(x[12]), __uint_as_float(x[13]));
          a = max3(a, __uint_as_float(x[14]), __uint_as_float(x[15]));
          m_cand = fmaxf(m_cand, fmaxf(a, d) * cg[q]);
        }
        const bool grow = m_cand > m_run + kChunkTau;
        const float m_new = grow ? m_cand : m_run;
        const float fac = grow ? ex2_approx(m_run - m_new) : 1.0f;  // 0 on the first tile
        m_run = m_new;
        const float m_use = m_run == -INFINITY ? 0.f : m_run;
        const float p_max = ex2_approx(m_cand - m_use);
        const float p_max_err = round_to_f16(p_max) - p_max;
        const uint64_t nm2 = f2_pack(-m_use, -m_use);
        uint64_t la = 0, lb = 0;
        uint32_t pk[64];
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          const uint64_t c2 = f2_pack(cg[i >> 3], cg[i >> 3]);
          float x0, x1, x2, x3;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2,
                           nm2),
                    x0, x1);
          f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * i + 2]), __uint_as_float(s[2 * i + 3])),
                           c2, nm2),
                    x2, x3);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          const float p2 = ex2_approx(x2), p3 = ex2_approx(x3);
          pk[i] = pack_f16x2(p0, p1);
          pk[i + 1] = pack_f16x2(p2, p3);
          la = f2_add(la, f2_pack(p0, p1));
          lb = f2_add(lb, f2_pack(p2, p3));
        }
        tmem_st_32x32b_x32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
        tmem_st_32x32b_x32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
        // the value tile this step multiplies, and its exponent
        if (!mbar_wait(&sb.v_ready[idx % C::kV16s], (idx / C::kV16s) & 1, abort_flag)) {
          chunk_abort(sb, p.err);
          goto done;
        }
        const int e_j = sb.v_exp[idx % C::kV16s];
        const float ofac = j == 0 || e_j == e_cur ? fac : fac * exp2i(max(e_j - e_cur, -126));
        e_cur = e_j;
        if (j > 0 && __any_sync(0xffffffffu, ofac != 1.0f)) {
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              reg_barrier(o[i]);
              reg_barrier(o[i + 1]);
              float a, d;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(o[i]), __uint_as_float(o[i + 1])),
                               f2_pack(ofac, ofac)),
                        a, d);
              o[i] = __float_as_uint(a);
              o[i + 1] = __float_as_uint(d);
            }
            tmem_st_32x32b_x32(tO + c0, o);
          }
        }
        {
          float a0, a1;
          f2_unpack(f2_add(la, lb), a0, a1);
          l_run = l_run * fac + (a0 + a1);
          lc_run = lc_run * fac + p_max_err;
        }
        if (j == n_t - 1) {
          sb.m_fin[part & 1][t][row] = m_run;
          sb.l_fin[part & 1][t][row] = l_run;
          sb.lc_fin[part & 1][t][row] = lc_run;
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sb.p_full[t]);
          if (j == n_t - 1) mbar_arrive(&sb.fin_full[part & 1][t]);
        }
      }
      ++part;
      step0 = step_end;
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ value conversion + epilogue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n" ::: "memory");
    const int cw = warp - 8;
    const int row = cw * 32 + lane;  // epilogue: row == TMEM lane
    const uint32_t lane_off = (uint32_t)(cw * 32) << 16;
    // conversion: eight lanes take rows x and x ^ 5 of eight, four pieces each:
    // neither the reads nor the writes of the swizzled tiles meet in a bank
    const int crow = (lane >> 3) ^ ((lane & 4) ? 5 : 0), cpiece = lane & 3;
    uint32_t step0 = 0, segs = 0;
    uint32_t part[2] = {0, 0};
    // the segment whose epilogue is pending
    bool pend = false;
    int pwhole = 0;
    int pb = 0, ph = 0, pmb = 0, pn[2] = {0, 0}, pe[2] = {0, 0}, prows = 0, plen = 0, pseg = 0;
#pragma unroll 1
    while (true) {
      ChunkSeg sg;
      if (!chunk_next(sb, segs, lane == 0, abort_flag, sg)) {
        chunk_abort(sb, p.err);
        goto done;
      }
      const bool have = sg.mb >= 0;
      const int n = have ? (kPair ? 2 * sg.n : sg.n) : 0;  // key tiles
      const int first = kPair ? 2 * sg.j0 : sg.j0;
      int e_run = 0, e_max = kKv8ExpMin, e_t0 = 0, e_t1 = 0;
#pragma unroll 1
      for (int j = 0; j <= n; ++j) {
        if (pend && (j == 1 || !have)) {
          // every converter warp has seen the segment's value codes
          if (!mbar_wait(&sb.conv_bar, (segs - 1) & 1, abort_flag)) {
            chunk_abort(sb, p.err);
            goto done;
          }
          const int par = (segs - 1) & 7;
          const bool nan = sb.nan_any[par] != 0;
          // the segment before is read by every converter warp: its slot starts anew
          sb.nan_pos[(par + 7) & 7][row] = 0x7fffffff;
          if (cw == 0 && lane == 0) sb.nan_any[(par + 7) & 7] = 0;
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            if (pn[t] == 0) continue;
            const uint32_t pc = part[t]++;
            if (!mbar_wait(&sb.fin_full[pc & 1][t], (pc >> 1) & 1, abort_flag) ||
                !mbar_wait(&sb.o_full[t], pc & 1, abort_flag)) {
              chunk_abort(sb, p.err);
              goto done;
            }
            tc_fence_after_sync();
            const float m = sb.m_fin[pc & 1][t][row];
            const float l = sb.l_fin[pc & 1][t][row];
            float oscale = exp2i(-pe[t]) / (l + sb.lc_fin[pc & 1][t][row]);
            if (l == 0.f) oscale = 0.f;  // no position seen (O is 0)
            float m2 = l == 0.f ? -INFINITY : m + lg2_approx(l);  // log2 of the sum
            const int r = kPair ? row : pmb * kChunkRows + t * 128 + row;
            const bool ok = r < prows * p.G;
            const int i = ok ? row_query(p, r) : 0;
            const int see = ok ? row_sees(p, i, plen, prows) : 0;
            const uint32_t tO = tmem + lane_off + (t ? C::kColO1 : C::kColO0);
            const long long orow =
                ((long long)pb * p.H + ph * p.G + (ok ? r - i * p.G : 0)) * p.Nq + i;
            float *part_row = p.part + (((size_t)blockIdx.x * 2 + (pseg > 0)) * kChunkRows +
                                        t * 128 + row) * (D + 4);
            // With pairs a whole unit's first tile is left in the slot (free until the
            // run's last segment), and joined with the second by the same thread.
            const bool join = kPair && pwhole && t == 1;
            const bool last = pwhole && (!kPair || t == 1);
            const float *other = part_row - 128 * (D + 4);
            float w_other = 0.f;
            if (join && ok) {
              const float mo = other[D], mm = fmaxf(mo, m2);
              const float a0 = other[D + 2] == 0.f ? 0.f : ex2_approx(mo - mm);
              const float a1 = l == 0.f ? 0.f : ex2_approx(m2 - mm), sum = a0 + a1;
              const float inv = sum == 0.f ? 0.f : 1.f / sum;
              oscale *= a1 * inv;
              w_other = a0 * inv;
              m2 = sum == 0.f ? -INFINITY : mm + lg2_approx(sum);
            }
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(tO + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                reg_barrier(o[k]);
                o[k] = __float_as_uint(__uint_as_float(o[k]) * oscale);
              }
              if (join && ok) {
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                  const float4 v = *reinterpret_cast<const float4 *>(other + c0 + k);
                  const float u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                  for (int z = 0; z < 4; ++z)
                    o[k + z] = __float_as_uint(fmaf(u[z], w_other, __uint_as_float(o[k + z])));
                }
              }
              if (ok && last) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.o + orow * D + c0);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  dst[k] = make_uint4(
                      pack_bf16x2(__uint_as_float(o[8 * k]), __uint_as_float(o[8 * k + 1])),
                      pack_bf16x2(__uint_as_float(o[8 * k + 2]), __uint_as_float(o[8 * k + 3])),
                      pack_bf16x2(__uint_as_float(o[8 * k + 4]), __uint_as_float(o[8 * k + 5])),
                      pack_bf16x2(__uint_as_float(o[8 * k + 6]), __uint_as_float(o[8 * k + 7])));
              } else if (ok) {
                uint4 *dst = reinterpret_cast<uint4 *>(part_row + c0);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
              }
            }
            if (ok) {
              if (last)
                p.lse[orow] = m2 * 0.69314718055994531f;
              else  // as merge_row takes it: O is normalised, so l is 1 or nothing
                *reinterpret_cast<float4 *>(part_row + D) =
                    make_float4(m2, m2 + kDecLift, l == 0.f ? 0.f : m2 == m2 ? 1.f : m2, 0.f);
              if (nan) {  // columns in which this row sees a NaN
#pragma unroll 1
                for (int k = 0; k < D; ++k)
                  if (sb.nan_pos[par][k] < see) {
                    if (last)
                      p.o[orow * D + k] = __ushort_as_bfloat16((unsigned short)0x7fc0u);
                    else
                      part_row[k] = __uint_as_float(0x7fc00000u);
                  }
              }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sb.o_free[t]);
          }
          pend = false;
        }
        if (j == n) break;
        // Convert one value tile.
        const uint32_t idx = step0 + j;
        const uint32_t vs = idx % C::kVs, ws = idx % C::kV16s;
        if (!mbar_wait(&sb.v_full[vs], (idx / C::kVs) & 1, abort_flag) ||
            (idx >= (uint32_t)C::kV16s &&
             !mbar_wait(&sb.v_free[ws], (idx / C::kV16s - 1) & 1, abort_flag))) {
          chunk_abort(sb, p.err);
          goto done;
        }
        const int v_valid = sb.v_valid[idx & 7];
        const int k0 = (first + j) * 128;
        {
          // (runs that could not be read carry the least exponent)
          int e8 = sb.v_exp8[idx & 7][lane & 7];
          e_max = max(e_max, __reduce_max_sync(0xffffffffu, e8));
        }
        e_run = kChunkLift - e_max;
        const uint8_t *raw = smem + C::kOffV + vs * C::kRaw;
        uint8_t *dst = smem + C::kOffV16 + ws * C::kV16;
        // 16 codes of row tr, piece pc, to fp16 times 2^(ve - E + lift)
        auto put = [&](int tr, int pc, const uint32_t(&x)[4]) {
          const float fs = exp2i(max(sb.v_exp8[idx & 7][tr >> 4] + e_run, -126));
          const uint32_t f2 = pack_f16x2(fs, fs);
          uint32_t o[8];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            e4m3x4_to_f16x2x2(x[y], o[2 * y], o[2 * y + 1]);
            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o[2 * y]) : "r"(f2));
            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o[2 * y + 1]) : "r"(f2));
          }
          uint8_t *line = dst + (pc >> 2) * 16384 + tr * 128;
          *reinterpret_cast<uint4 *>(line + (((2 * (pc & 3)) ^ (tr & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4 *>(line + (((2 * (pc & 3) + 1) ^ (tr & 7)) << 4)) =
              make_uint4(o[4], o[5], o[6], o[7]);
        };
        auto get = [&](int tr, int pc) {
          if constexpr (D == 128)
            return *reinterpret_cast<const uint4 *>(raw + tr * 128 + ((pc ^ (tr & 7)) << 4));
          else
            return *reinterpret_cast<const uint4 *>(raw + tr * 64 + ((pc ^ ((tr >> 1) & 3)) << 4));
        };
        uint32_t any = 0;
        auto convert = [&](int tr, int pc, const uint4 &w) {
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) any |= (x[y] & 0x7f7f7f7fu) + 0x01010101u;
          put(tr, pc, x);
        };
        if constexpr (kPair) {
          static_assert(!kPair || D == 64, "one piece of a row a read");
          // Two tiles a step, short rows: all of a lane's reads in flight (110 -> 85 us
          // for 32 sequences of up to 32768 positions, 48 rows a head).
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = get(cw * 32 + i * 8 + crow, cpiece);
#pragma unroll
          for (int i = 0; i < 4; ++i) convert(cw * 32 + i * 8 + crow, cpiece, w[i]);
        } else {
          // (Unrolled at D = 128 it takes more of the instruction fetch and of the
          // registers than it gives: 430 -> 530 us at 2048 x 16384.)
#pragma unroll 1
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int hc = 0; hc < D / 64; ++hc) {
              const int tr = cw * 32 + i * 8 + crow, pc = hc * 4 + cpiece;
              convert(tr, pc, get(tr, pc));
            }
        }
        // Rows past the length or without a page, and NaN codes: this lane's
        // pieces once more, with zeros in their place.
        if (v_valid != 0xff || k0 + 128 > sg.len || (any & 0x80808080u)) {
#pragma unroll 1
          for (int z = 0; z < D / 16; ++z) {
            const int tr = cw * 32 + (z / (D / 64)) * 8 + crow, pc = (z % (D / 64)) * 4 + cpiece;
            const uint4 w = get(tr, pc);
            uint32_t x[4] = {w.x, w.y, w.z, w.w};
            const bool off = !(v_valid >> (tr >> 4) & 1) || k0 + tr >= sg.len;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t hit = ((x[y] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              if (off) hit = 0x80808080u;
              x[y] &= ~((hit >> 7) * 0xffu);
              if (!off && hit) {
                sb.nan_any[segs & 7] = 1;
#pragma unroll 1
                for (int k = 0; k < 4; ++k)
                  if (hit >> (8 * k + 7) & 1)
                    atomicMin(&sb.nan_pos[segs & 7][pc * 16 + 4 * y + k], k0 + tr);
              }
            }
            put(tr, pc, x);
          }
          __syncwarp();
        }
        fence_proxy_async_smem();
        if (cw == 0 && lane == 0) sb.v_exp[ws] = e_run;
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sb.v_ready[ws]);
          mbar_arrive(&sb.v_empty[vs]);
        }
        if (j == (kPair ? n - 2 : sg.n0 - 1)) e_t0 = e_run;
        if (j == (kPair ? n - 1 : sg.n1 - 1)) e_t1 = e_run;
      }
      if (!have) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb.conv_bar);
      pend = true;
      pwhole = sg.whole;
      pb = sg.b;
      ph = sg.h;
      pmb = sg.mb;
      pn[0] = sg.n0;
      pn[1] = sg.n1;
      pe[0] = e_t0;
      pe[1] = e_t1;
      prows = sg.rows;
      plen = sg.len;
      pseg = (int)segs;
      ++segs;
      step0 += n;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n" ::: "memory");
    if (warp == 12 && lane == 0) {
      // ---------------------------------------------------------- tensor-core issue
      // Step j: P0 V_{j-1}, S0 = Q0 K_j^T, then P1 V_{j-1}, S1 = Q1 K_j^T, so each
      // tile's softmax works while the other tile's products run.
      constexpr uint32_t idS = idesc_e4m3_f32(128, 128);
      constexpr uint32_t idO = idesc_f32acc(false, 128, D, false, true);
      const uint32_t hi128 = sdesc_sw128_hi(1024);
      const uint32_t hik = D == 128 ? sdesc_sw128_hi(1024) : sdesc_sw64_hi(512);
      const uint32_t q_lo0 = sdesc_sw128_lo(smem_addr(smem), 16);
      const uint32_t k_lo0 = sdesc_sw128_lo(smem_addr(smem + C::kOffK), 16);
      const uint32_t v_lo0 = sdesc_sw128_lo(smem_addr(smem + C::kOffV16), 16384);
      // One body for both tiles (the other roles take most of the instruction
      // fetch), its products unrolled: a rolled issue loop took 95 cycles a
      // product, where the tensor core takes 64.
      uint32_t p_phase = 0;            // bit t
      uint32_t parts = 0, started = 0; // bit t: parity of segments done, any done
      uint32_t ks = 0, k_turn = 0;     // key ring slot of step j, parity of its use
      uint32_t ws = 0;                 // fp16 value slot of step j - 1
#pragma unroll 1
      for (uint32_t sx = 0;; ++sx) {
        ChunkSeg sg;
        if (!chunk_next(sb, sx, true, abort_flag, sg)) {
          chunk_abort(sb, p.err);
          goto mma_exit;
        }
        if (sg.mb < 0) break;
        const int n = sg.n, n0 = sg.n0, n1 = sg.n1;
#pragma unroll 1
        for (int j = 0; j <= n; ++j) {
          bool k_ready = false;
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            const int n_t = t ? n1 : n0;
            const bool do_pv = j >= 1 && j <= n_t;
            const bool do_s = j < n_t;
            const uint32_t tS = tmem + t * (C::kColS1 - C::kColS0);
            const uint32_t tO = tmem + C::kColO0 + t * (C::kColO1 - C::kColO0);
            if (do_pv) {
              // (P is signalled only once V_{j-1} is converted)
              if ((j == 1 && (started >> t & 1) &&
                   !mbar_wait(&sb.o_free[t], ~(parts >> t) & 1, abort_flag)) ||
                  !mbar_wait(&sb.p_full[t], p_phase >> t & 1, abort_flag)) {
                chunk_abort(sb, p.err);
                goto mma_exit;
              }
              p_phase ^= 1u << t;
            }
            if (do_s) {
              if ((j == 0 && !mbar_wait(&sb.q_full[t], parts >> t & 1, abort_flag)) ||
                  (!k_ready && !mbar_wait(&sb.k_full[ks], k_turn, abort_flag))) {
                chunk_abort(sb, p.err);
                goto mma_exit;
              }
              k_ready = true;
            }
            tc_fence_after_sync();
            if (do_pv) {
              const uint32_t v_lo = v_lo0 + (kPair ? t : ws) * (C::kV16 >> 4);
              umma_ts_w_rt(tO, tS, v_lo, hi128, idO, j > 1 ? 1u : 0u);
#pragma unroll
              for (int kk = 1; kk < 8; ++kk)
                umma_ts_w<1>(tO, tS + kk * 8, v_lo + kk * (2048 >> 4), hi128, idO);
            }
            if (do_s) {
              // 32 codes a product; hi, then lo
              const uint32_t a = q_lo0 + t * (C::kQTile >> 4), bk = k_lo0 + ks * (C::kRaw >> 4);
              umma_f8_ss<0>(tS, a, hi128, bk, hik, idS);
#pragma unroll
              for (int kk = 1; kk < D / 16; ++kk) {
                const int x = kk % (D / 32);
                const uint32_t off =
                    D == 128 ? (kk / 4) * (16384 >> 4) + x * 2 : (uint32_t)kk * 2;
                umma_f8_ss<1>(tS, a + off, hi128, bk + x * 2, hik, idS);
              }
              umma_commit(&sb.s_full[t]);
            }
            if constexpr (kPair) {  // each tile has its own key and value tiles
              if (do_pv) umma_commit(&sb.v_free[t]);
              if (do_s) {
                umma_commit(&sb.k_empty[ks]);
                k_ready = false;
                if (++ks == C::kKs) {
                  ks = 0;
                  k_turn ^= 1;
                }
              }
            }
            if (do_pv && j == n_t) {
              umma_commit(&sb.o_full[t]);
              parts ^= 1u << t;
              started |= 1u << t;
            }
          }
          if constexpr (!kPair) {
            if (j < n) {
              umma_commit(&sb.k_empty[ks]);
              if (++ks == C::kKs) {
                ks = 0;
                k_turn ^= 1;
              }
            }
            if (j >= 1) {
              umma_commit(&sb.v_free[ws]);
              ws ^= 1;
            }
          }
        }
      }
    mma_exit:
      // every product must finish before the tensor memory is freed
      umma_commit(&sb.mma_done);
      {
        int never = 0;
        mbar_wait(&sb.mma_done, 0, &never);
      }
    }
    if (warp == 15) {
      // ---------------------------------------------------------- the run's segments
      const long long share = sb.place.share;
      const long long u0 = blockIdx.x * share;
      long long left = max(0LL, min(share, sb.place.total - u0));
      int b = sb.place.b, h = 0, mb = 0, j = 0;
      ChunkSeq q = {0, 0, 0};
      if (left > 0) {
        // where the run starts: the head, then the unit, 32 units at a time
        q = chunk_seq(p, b);
        const long long per_head = chunk_seq_cost_warp(p, b, lane);
        long long r = u0 - sb.place.prefix;
        h = (int)(r / per_head);
        r -= h * per_head;
#pragma unroll 1
        for (int m0 = 0;; m0 += 32) {
          const int c = m0 + lane < q.units ? chunk_cost(p, q, m0 + lane) : 0;
          int inc = c;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += t;
          }
          const uint32_t in = __ballot_sync(0xffffffffu, r < inc);
          if (in != 0 || m0 + 32 >= q.units) {
            const int at = in != 0 ? __ffs(in) - 1 : 31;  // (always found)
            mb = m0 + at;
            j = (int)(r - __shfl_sync(0xffffffffu, inc - c, at));
            break;
          }
          r -= __shfl_sync(0xffffffffu, inc, 31);
        }
      }
      if (lane != 0) left = 0;  // one thread posts them
#pragma unroll 1
      for (uint32_t x = 0; lane == 0; ++x) {
        if (x >= 4 && !mbar_wait(&sb.seg_empty[x & 3], ((x >> 2) - 1) & 1, abort_flag)) {
          chunk_abort(sb, p.err);
          break;
        }
        ChunkSeg &sg = sb.seg[x & 3];
        if (left == 0) {
          sg.mb = -1;
          mbar_arrive(&sb.seg_full[x & 3]);
          break;
        }
        const int cost = chunk_cost(p, q, mb);
        const int t0 = kPair ? cost : chunk_tiles(p, mb * kChunkRows, q.len, q.rows);
        const int t1 = kPair ? cost : chunk_tiles(p, mb * kChunkRows + 128, q.len, q.rows);
        const int n = (int)min((long long)(cost - j), left);
        sg.b = b;
        sg.h = h;
        sg.mb = mb;
        sg.j0 = j;
        sg.n = n;
        sg.n0 = min(max(t0 - j, 0), n);
        sg.n1 = min(max(t1 - j, 0), n);
        sg.len = q.len;
        sg.rows = q.rows;
        sg.whole = j == 0 && n == cost;
        mbar_arrive(&sb.seg_full[x & 3]);
        left -= n;
        j += n;
        if (j == cost) {
          j = 0;
          if (++mb == q.units) {
            mb = 0;
            if (++h == g.Hkv) {
              h = 0;
#pragma unroll 1
              while (++b < p.B) {
                q = chunk_seq(p, b);
                if (q.units > 0) break;
              }
            }
          }
        }
      }
    }
    if (warp == 13 || warp == 14)
      chunk_load<D, kPair>(p, warp == 13, warp == 13 ? &tm_v : &tm_k, sb,
                    smem + (warp == 13 ? C::kOffV : C::kOffK), lane, abort_flag);
  }
done:
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 12) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// Where a row's partials lie: n of them (0: one run held the unit whole), from
// run c0 on, c0's in its slot `first`; with pairs two a run.  `before` and `all`:
// steps of the head's units before the row's, and of all of them (after grid_wait).
struct ChunkParts {
  int c0, n, first, pair;
  __device__ __forceinline__ size_t row(int k, int r) const {  // of the partials' rows
    const int c = pair ? k >> 1 : k;
    return ((size_t)(c0 + c) * 2 + (c == 0 ? first : 0)) * kChunkRows + r % kChunkRows +
           (pair ? (k & 1) * 128 : 0);
  }
};
__device__ __forceinline__ ChunkParts chunk_parts(const Kv8AttnParams &p, const ChunkSeq &s, int b,
                                                  int h, int r, long long before,
                                                  long long all) {
  const long long share = p.prefix[p.B];
  const long long s0 = p.prefix[b] + h * all + before;
  ChunkParts a;
  a.pair = p.pair;
  a.c0 = (int)(s0 / share);
  a.first = a.c0 * share == s0 ? 0 : 1;
  const int c1 = (int)((s0 + chunk_cost(p, s, r / kChunkRows) - 1) / share);
  if (c1 == a.c0) {
    a.n = 0;
  } else if (p.pair) {
    a.n = 2 * (c1 - a.c0 + 1);
  } else {  // runs that hold no key tile of the row's tile wrote nothing for it
    const int tiles = chunk_tiles(p, r / 128 * 128, s.len, s.rows);
    a.n = min(c1, (int)((s0 + tiles - 1) / share)) - a.c0 + 1;
  }
  return a;
}

// Steps of a head's units before unit mb, and of all: a warp.
__device__ __forceinline__ void chunk_before(const Kv8AttnParams &p, const ChunkSeq &s, int mb,
                                             int lane, long long &before, long long &all) {
  before = all = 0;
#pragma unroll 1
  for (int x = lane; x < s.units; x += 32) {
    const int c = chunk_cost(p, s, x);
    all += c;
    if (x < mb) before += c;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, d);
    all += __shfl_xor_sync(0xffffffffu, all, d);
  }
}

// Merge where units lie in many runs: a block a row.  grid: (Nq * G, Hkv, B)
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    tk_kv8_chunk_merge_deep_kernel(const __grid_constant__ Kv8AttnParams p) {
  const int r = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const ChunkSeq s = chunk_seq(p, b);
  const int mb = r / kChunkRows;
  long long before, all;
  chunk_before(p, s, mb, threadIdx.x & 31, before, all);
  grid_wait();  // (above: only what the launch before leaves alone)
  if (r >= s.rows * p.G) return;
  const ChunkParts at = chunk_parts(p, s, b, h, r, before, all);
  if (at.n == 0) return;
  const int i = row_query(p, r);
  const long long orow = ((long long)b * p.H + h * p.G + (r - i * p.G)) * p.Nq + i;
  merge_row<D>([&](int k) { return p.part + at.row(k, r) * (D + 4); }, at.n, p.o + orow * D,
               p.lse + orow);
}

// Merge where units lie in few runs: a warp takes four rows of one tile, all
// their partials of a run in flight together.  grid: (ceil(Nq * G / 32), Hkv, B)
constexpr int kChunkMergeRows = 4;
template <int D>
__global__ void __launch_bounds__(256)
    tk_kv8_chunk_merge_kernel(const __grid_constant__ Kv8AttnParams p) {
  constexpr int kPer = D / 32;
  const int b = blockIdx.z, h = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int r0 = blockIdx.x * (8 * kChunkMergeRows) + (threadIdx.x >> 5) * kChunkMergeRows;
  const ChunkSeq s = chunk_seq(p, b);
  const int mb = r0 / kChunkRows, r_end = s.rows * p.G;
  long long before, all;
  chunk_before(p, s, mb, lane, before, all);
  grid_wait();  // (above: only what the launch before leaves alone)
  if (r0 >= r_end) return;
  const ChunkParts at = chunk_parts(p, s, b, h, r0, before, all);
  if (at.n == 0) return;
  float mx[kChunkMergeRows], z[kChunkMergeRows], acc[kChunkMergeRows][kPer];
#pragma unroll
  for (int i = 0; i < kChunkMergeRows; ++i) {
    mx[i] = kDecNone;
    z[i] = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[i][k] = 0.f;
  }
#pragma unroll 2
  for (int c = 0; c < at.n; ++c) {
    const float *d = p.part + at.row(c, r0) * (D + 4);
    float l[kChunkMergeRows], x[kChunkMergeRows][kPer];
#pragma unroll
    for (int i = 0; i < kChunkMergeRows; ++i) {
      l[i] = -INFINITY;
#pragma unroll
      for (int k = 0; k < kPer; ++k) x[i][k] = 0.f;
      if (r0 + i < r_end) {
        l[i] = d[i * (D + 4) + D];  // log2 of the run's sum
#pragma unroll
        for (int k = 0; k < kPer; ++k) x[i][k] = d[i * (D + 4) + lane * kPer + k];
      }
    }
#pragma unroll
    for (int i = 0; i < kChunkMergeRows; ++i) {
      const float m = fmaxf(mx[i], l[i]);
      const float up = exp2f(mx[i] - m), w = exp2f(l[i] - m);  // (l none: 0; NaN stays)
      mx[i] = m;
      z[i] = fmaf(z[i], up, w);
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[i][k] = fmaf(w, x[i][k], acc[i][k] * up);
    }
  }
#pragma unroll
  for (int i = 0; i < kChunkMergeRows; ++i) {
    const int r = r0 + i;
    if (r >= r_end) break;
    const float inv = z[i] == 0.f ? 0.f : 1.f / z[i];
    const int n = row_query(p, r);
    const long long orow = ((long long)b * p.H + h * p.G + (r - n * p.G)) * p.Nq + n;
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.o + orow * D + lane * kPer);
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k)
      dst[k] = pack_bf16x2(acc[i][2 * k] * inv, acc[i][2 * k + 1] * inv);
    if (lane == 0) p.lse[orow] =
          z[i] == 0.f ? -INFINITY : (mx[i] + log2f(z[i])) * 0.69314718055994531f;
  }
}

}  // namespace tkattn
