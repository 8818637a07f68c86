// tk_norm_rope.cu -- RMS norm of each head's query and key with the position
// rotation in the same pass, forward and backward.
//
// For every head row x (D values) of a token at position p:
//   n = x * r,  r = (mean(x^2) + eps)^(-1/2);   y = R(p) (n o w)
// R(p) turns the pairs (a, b) of the row's first `rot` values by the angles
// p f_k:  (a, b) -> (a cos - b sin, b cos + a sin); pair k is (k, rot/2 + k),
// or (2k, 2k+1) when interleaved; the values past `rot` pass unturned.
// Backward, with g = R(p)^T dy:
//   dx = r (g o w - n mean(g o w o n)),   dw = sum over rows of g o n.
//
// Angles: a frequency is given in turns a position as a 64-bit fraction F of
// one turn, so p F modulo 2^64 is the exact fraction of a turn at any 32-bit
// position: no reduction, no loss at far positions.  Its top 32 bits, rounded
// to fp32, go to sincospif.
//
// Mapping: D/8 lanes own a head row, eight values each, in two groups of four
// placed so that a pair's two values sit in one lane (no exchange for the
// rotation; three or four shuffles for the mean).  A row group keeps one
// token's sines and cosines, multiplied by the weights, for `hpg` consecutive
// heads; the groups of a block take consecutive tokens, so a block writes runs
// of consecutive rows of a head-major output.
// Everything is computed in fp32 and rounded once to bf16.
//
// Bound by bytes: 4 x 4096 tokens of 32 + 8 heads of 128 take 54 us (335 MB, 6.2
// TB/s).  What an SM needs is loads outstanding while other rows are reduced: 28 to
// 32 warps with four rows each, in small blocks, so that few wait for a block's
// last (with 128 threads 56 us, and 1 x 4096 tokens 16.5 for 15.1).  16 x 1024
// tokens of 16 + 16 heads of 64, forward and gradients, take 61 us: 22 + 39, 5.5
// TB/s over the five tensors of 67 MB that the two calls read and write.  One token
// for each of 8 sequences takes 2.2 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <utility>

#include "sm103_ptx.cuh"
#include "tk_attn.h"
#include "tk_device.h"
#include "tk_launch.cuh"

namespace tkattn {
namespace {

constexpr int kNrFwdThreads = 64, kNrBwdThreads = 256;
// Forward: blocks of an SM.  72 registers hold the paired halves' kernel, in 64 it
// spills (4 x 4096 tokens, 40 heads of 128: 59.4 us; 65 with 12 blocks); the other fits 64.
template <bool kHalves>
constexpr int kNrFwdBlocks = kHalves ? 14 : 16;
// Backward: blocks of an SM, and heads whose rows are loaded together, the next ones
// while these are worked on (without that 16 x 1024 tokens, 32 heads of 64, took
// with the forward 62.7 us for 61.3 and four heads at a time on two blocks).
constexpr int kNrBwdBlocks = 3, kNrBwdUnroll = 2;
constexpr int kNrFwdHeads = 32, kNrBwdHeads = 8;  // heads a row group takes for one token, at most
// Rows of partial weight gradients: one for each block of the backward.
constexpr int kNrBwdMaxBlocks = 2048;

struct NrTensor {
  const __nv_bfloat16 *p;
  long long sb, sh, sn;  // element strides of batch, head, token
};

struct NrParams {
  NrTensor x[2];    // queries, keys
  NrTensor dy[2];   // backward: gradients of the outputs
  __nv_bfloat16 *y[2];
  long long yb[2], yh[2], yn[2];  // element strides of the results
  const void *w[2];
  int w_f32;
  const uint64_t *turns;
  const int *pos;  // [B, N] or null: 0 .. N-1
  float eps;
  int B, N, H[2], rot;
  int hpg;          // heads a row group takes for one token
  int chunks[2];    // ceil(H / hpg): gridDim.y of the two together
  int tiles;        // ceil(B * N / groups per block)
  int early;        // the next grid may begin beside this one (tk_launch.cuh)
  float *dw_part;   // [gridDim.y * gridDim.x, D]: the queries' rows, then the keys'
};

// First columns of a lane's two groups of four: pair i is (lo + i, hi + i) when
// halves are paired; neighbours when interleaved; past the rotated values
// eight in a row either way.
__device__ __forceinline__ void lane_cols(int l, int rot, bool halves, int &lo, int &hi) {
  if (halves && l < rot / 8) {
    lo = 4 * l;
    hi = rot / 2 + 4 * l;
  } else {
    lo = 8 * l;
    hi = 8 * l + 4;
  }
}

struct Raw {  // eight bf16 values as loaded
  uint2 lo, hi;
};

template <bool kHalves>
__device__ __forceinline__ Raw load8(const __nv_bfloat16 *row, int lo, int hi) {
  Raw r;
  if constexpr (kHalves) {
    r.lo = __ldg(reinterpret_cast<const uint2 *>(row + lo));
    r.hi = __ldg(reinterpret_cast<const uint2 *>(row + hi));
  } else {  // eight in a row
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(row + lo));
    r.lo = make_uint2(v.x, v.y);
    r.hi = make_uint2(v.z, v.w);
  }
  return r;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The lane's four pairs (a, b): across the two groups, or neighbours.
template <bool kHalves>
__device__ __forceinline__ void pairs_of(const Raw &r, float (&a)[4], float (&b)[4]) {
  if constexpr (kHalves) {
    a[0] = bf_lo(r.lo.x), a[1] = bf_hi(r.lo.x), a[2] = bf_lo(r.lo.y), a[3] = bf_hi(r.lo.y);
    b[0] = bf_lo(r.hi.x), b[1] = bf_hi(r.hi.x), b[2] = bf_lo(r.hi.y), b[3] = bf_hi(r.hi.y);
  } else {
    a[0] = bf_lo(r.lo.x), b[0] = bf_hi(r.lo.x), a[1] = bf_lo(r.lo.y), b[1] = bf_hi(r.lo.y);
    a[2] = bf_lo(r.hi.x), b[2] = bf_hi(r.hi.x), a[3] = bf_lo(r.hi.y), b[3] = bf_hi(r.hi.y);
  }
}

template <bool kHalves>
__device__ __forceinline__ void store8(__nv_bfloat16 *row, int lo, int hi, const float (&a)[4],
                                       const float (&b)[4]) {
  if constexpr (kHalves) {
    *reinterpret_cast<uint2 *>(row + lo) =
        make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
    *reinterpret_cast<uint2 *>(row + hi) =
        make_uint2(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]));
  } else {
    *reinterpret_cast<uint4 *>(row + lo) =
        make_uint4(pack_bf16x2(a[0], b[0]), pack_bf16x2(a[1], b[1]), pack_bf16x2(a[2], b[2]),
                   pack_bf16x2(a[3], b[3]));
  }
}

// Column of a lane's value i of the first (a) or second (b) of its pairs.
template <bool kHalves>
__device__ __forceinline__ int pair_col(int lo, int hi, int i, int second) {
  if constexpr (kHalves) return (second ? hi : lo) + i;
  return (i < 2 ? lo : hi) + 2 * (i & 1) + second;
}

__device__ __forceinline__ float weight_at(const void *w, int f32, int c) {
  return f32 ? static_cast<const float *>(w)[c]
             : __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[c]);
}

// cos and sin of a lane's four pairs at position p.
__device__ __forceinline__ void lane_angles(const uint64_t *turns, int l, int p, bool on,
                                            float (&cs)[4], float (&sn)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  if (!on) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t frac = (uint64_t)(long long)p * turns[4 * l + i];
    // signed 32-bit fraction: half turns in [-1, 1)
    const float half_turns = (float)(int)(frac >> 32) * 4.656612873077393e-10f;  // 2^-31
    sincospif(half_turns, &sn[i], &cs[i]);
  }
}

template <int kLanes>
__device__ __forceinline__ float group_sum(float s) {
#pragma unroll
  for (int d = kLanes / 2; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}

// grid: (token tiles, or fewer blocks that step over them; runs of hpg heads,
// the queries' first).  A block takes one token for each of its row groups.
template <int D, bool kHalves, bool kBwd>
__global__ void __launch_bounds__(kBwd ? kNrBwdThreads : kNrFwdThreads,
                                  kBwd ? kNrBwdBlocks : kNrFwdBlocks<kHalves>)
    tk_norm_rope_kernel(const __grid_constant__ NrParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = (kBwd ? kNrBwdThreads : kNrFwdThreads) / kLanes;
  constexpr int kUnroll = kBwd ? kNrBwdUnroll : 4;  // heads whose rows are loaded together
  const int l = threadIdx.x % kLanes;
  const int grp = threadIdx.x / kLanes;
  int lo, hi;
  lane_cols(l, p.rot, kHalves, lo, hi);
  const bool turned = 8 * l < p.rot;
  const int which = (int)blockIdx.y >= p.chunks[0];
  const int h0 = ((int)blockIdx.y - (which ? p.chunks[0] : 0)) * p.hpg;
  const int h1 = min(h0 + p.hpg, p.H[which]);
  grid_launch_dependents_if(p.early);
  grid_wait();
  const NrTensor X = p.x[which];
  const long long yh = p.yh[which];
  float wa[4], wb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wa[i] = weight_at(p.w[which], p.w_f32, pair_col<kHalves>(lo, hi, i, 0));
    wb[i] = weight_at(p.w[which], p.w_f32, pair_col<kHalves>(lo, hi, i, 1));
  }
  float da[4] = {0.f, 0.f, 0.f, 0.f}, db[4] = {0.f, 0.f, 0.f, 0.f};  // backward: sums of g o n
  const unsigned tokens = (unsigned)p.B * (unsigned)p.N;
  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const unsigned tok = (unsigned)tile * kGroups + grp;
    const bool live = tok < tokens;
    const int b = live ? (int)(tok / (unsigned)p.N) : 0;
    const int n = live ? (int)(tok - (unsigned)b * (unsigned)p.N) : 0;
    const __nv_bfloat16 *xrow = X.p + b * X.sb + n * X.sn + h0 * X.sh;
    __nv_bfloat16 *yrow = p.y[which] + b * p.yb[which] + n * p.yn[which] + h0 * yh;
    const int end = live ? h1 - h0 : 0;  // heads this group has
    float cs[4], sn[4];
    lane_angles(p.turns, l, p.pos ? p.pos[live ? tok : 0] : n, turned, cs, sn);
    if constexpr (!kBwd) {
      // y_a = r (a wa cos - b wb sin), y_b = r (b wb cos + a wa sin)
      float ca[4], sa[4], cb[4], sb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ca[i] = wa[i] * cs[i];
        sa[i] = wa[i] * sn[i];
        cb[i] = wb[i] * cs[i];
        sb[i] = -wb[i] * sn[i];
      }
      for (int h = 0; h < h1 - h0; h += kUnroll) {
        Raw x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          x[u].lo = x[u].hi = make_uint2(0, 0);
          if (h + u < end) x[u] = load8<kHalves>(xrow + u * X.sh, lo, hi);
        }
        xrow += kUnroll * X.sh;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          float a[4], c[4];
          pairs_of<kHalves>(x[u], a, c);
          float ss = 0.f, s2 = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ss = fmaf(a[i], a[i], ss);
            s2 = fmaf(c[i], c[i], s2);
          }
          ss = group_sum<kLanes>(ss + s2);
          const float r = rsqrtf(fmaf(ss, 1.f / D, p.eps));
          float ya[4], yb[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ya[i] = fmaf(a[i], ca[i], c[i] * sb[i]) * r;
            yb[i] = fmaf(c[i], cb[i], a[i] * sa[i]) * r;
          }
          if (h + u < end) store8<kHalves>(yrow + u * yh, lo, hi, ya, yb);
        }
        yrow += kUnroll * yh;
      }
    } else {
      // The next heads' rows are on their way while these are worked on.
      const NrTensor G = p.dy[which];
      const __nv_bfloat16 *grow = G.p + b * G.sb + n * G.sn + h0 * G.sh;
      auto load = [&](Raw(&x)[kUnroll], Raw(&y)[kUnroll], int h) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          x[u].lo = x[u].hi = y[u].lo = y[u].hi = make_uint2(0, 0);
          if (h + u < end) {
            x[u] = load8<kHalves>(xrow + u * X.sh, lo, hi);
            y[u] = load8<kHalves>(grow + u * G.sh, lo, hi);
          }
        }
        xrow += kUnroll * X.sh;
        grow += kUnroll * G.sh;
      };
      auto work = [&](const Raw(&x)[kUnroll], const Raw(&y)[kUnroll], int h) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          float a[4], c[4], ga[4], gb[4];
          pairs_of<kHalves>(x[u], a, c);
          pairs_of<kHalves>(y[u], ga, gb);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // the rotation's transpose
            const float ta = fmaf(ga[i], cs[i], gb[i] * sn[i]);
            const float tb = fmaf(gb[i], cs[i], -ga[i] * sn[i]);
            ga[i] = ta;
            gb[i] = tb;
            ss = fmaf(a[i], a[i], fmaf(c[i], c[i], ss));
            dot = fmaf(ta * wa[i], a[i], fmaf(tb * wb[i], c[i], dot));
          }
          ss = group_sum<kLanes>(ss);
          dot = group_sum<kLanes>(dot);
          // dx = r g w - x r^3 mean(g w x)
          // (a group without a row adds nothing, whatever eps is)
          const float r = h + u < end ? rsqrtf(fmaf(ss, 1.f / D, p.eps)) : 0.f;
          const float back = dot * (1.f / D) * r * r * r;
          float va[4], vb[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ga[i] *= r;
            gb[i] *= r;
            da[i] = fmaf(ga[i], a[i], da[i]);
            db[i] = fmaf(gb[i], c[i], db[i]);
            va[i] = fmaf(ga[i], wa[i], -a[i] * back);
            vb[i] = fmaf(gb[i], wb[i], -c[i] * back);
          }
          if (h + u < end) store8<kHalves>(yrow + u * yh, lo, hi, va, vb);
        }
        yrow += kUnroll * yh;
      };
      Raw x0[kUnroll], y0[kUnroll], x1[kUnroll], y1[kUnroll];
      load(x0, y0, 0);
      for (int h = 0; h < h1 - h0; h += 2 * kUnroll) {
        load(x1, y1, h + kUnroll);
        work(x0, y0, h);
        if (h + kUnroll >= h1 - h0) break;
        load(x0, y0, h + 2 * kUnroll);
        work(x1, y1, h + kUnroll);
      }
    }
  }
  if constexpr (kBwd) {
    // the block's sums, in a fixed order
    __shared__ float part[kGroups][D];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      part[grp][pair_col<kHalves>(lo, hi, i, 0)] = da[i];
      part[grp][pair_col<kHalves>(lo, hi, i, 1)] = db[i];
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) s += part[g][threadIdx.x];
      p.dw_part[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * D + threadIdx.x] = s;
    }
  }
}

// dw = sum over the blocks' partial rows, in a fixed order: a block for 32
// columns of one weight, 32 warps over the rows, then over the warps.  Started
// while the launch before ends.  grid: (D / 32, 2)
__global__ void __launch_bounds__(1024)
    tk_norm_rope_dw_kernel(const float *__restrict__ part, int q_rows, int k_rows, int D,
                           float *__restrict__ dqw, float *__restrict__ dkw) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const int rows = blockIdx.y ? k_rows : q_rows;
  const float *base = part + (blockIdx.y ? (size_t)q_rows * D : 0) + col;
  grid_launch_dependents();
  grid_wait();
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r = warp; r < rows; r += 128) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r + 32 * i < rows) s[i] += base[(size_t)(r + 32 * i) * D];
  }
  acc[warp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (warp == 0) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += acc[i][lane];
    (blockIdx.y ? dkw : dqw)[col] = t;
  }
}

// (the stride of a dimension of one says nothing)
bool strides_ok(const long long *s, int B, int H, int N) {
  const int len[3] = {B, H, N};
  for (int i = 0; i < 3; ++i)
    if (len[i] == 1)
      continue;
    else if (s[i] < 0 || s[i] % 8 || s[i] >= (1LL << 40)) return false;
  return true;
}

// Bytes from a tensor's first to past its last element.
size_t extent(const long long *s, int B, int H, int N, int D) {
  return 2 * (size_t)((B - 1) * s[0] + (H - 1) * s[1] + (N - 1) * s[2] + D);
}

// A written tensor must not hold one element twice: every dimension longer
// than one has to step over the dimensions inside it.
bool distinct(const long long *s, int B, int H, int N, int D) {
  struct {
    long long stride, len;
  } d[3] = {{s[0], B}, {s[1], H}, {s[2], N}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (d[j].stride < d[i].stride) std::swap(d[i], d[j]);
  long long inner = D;
  for (auto &x : d) {
    if (x.len <= 1) continue;
    if (x.stride < inner) return false;
    inner = x.stride * (x.len - 1) + inner;
  }
  return true;
}

// Two written tensors whose extents overlap share no element: both lie in one
// token-major buffer (the same token and batch strides), their heads in
// disjoint runs of a token's values.
bool interleave_apart(uintptr_t a, const long long *sa, int Ha, uintptr_t b, const long long *sb,
                      int Hb, int B, int N, int D) {
  if ((b > a ? b - a : a - b) % 2) return false;
  long long period;  // elements from one token's values to the next's
  if (N > 1) {
    period = sa[2];
    if (sa[2] != sb[2] || period <= 0) return false;
    if (B > 1 && (sa[0] != sb[0] || sa[0] % period)) return false;
  } else {
    period = B > 1 ? sa[0] : 0;
    if (period <= 0 || sa[0] != sb[0]) return false;
  }
  const long long wa = (Ha - 1) * sa[1] + D, wb = (Hb - 1) * sb[1] + D;
  const long long off = ((long long)b - (long long)a) / 2;
  const long long r = ((off % period) + period) % period;
  return r >= wa && r + wb <= period;
}

struct Call {
  const void *q, *k, *qw, *kw;
  const long long *qs, *ks;
  const unsigned long long *turns;
  const int *positions;
  int B, H, Hk, N, D, rot, w_f32;
  float eps;
};

int check_common(const Call &c) {
  if (!c.q || !c.k || !c.qw || !c.kw || !c.qs || !c.ks) return TK_ATTN_ERR_INVALID_ARG;
  if (c.B <= 0 || c.H <= 0 || c.Hk <= 0 || c.N <= 0 || c.rot < 0 || c.rot > c.D)
    return TK_ATTN_ERR_INVALID_ARG;
  if (c.rot > 0 && !c.turns) return TK_ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(c.eps) || c.eps < 0.f) return TK_ATTN_ERR_INVALID_ARG;
  if ((c.D != 64 && c.D != 128) || c.rot % 8) return TK_ATTN_ERR_UNSUPPORTED;
  if (((uintptr_t)c.q | (uintptr_t)c.k) & 15u) return TK_ATTN_ERR_UNSUPPORTED;
  if ((uintptr_t)c.turns & 7u || (uintptr_t)c.positions & 3u ||
      ((uintptr_t)c.qw | (uintptr_t)c.kw) & (c.w_f32 ? 3u : 1u))
    return TK_ATTN_ERR_UNSUPPORTED;
  if (!strides_ok(c.qs, c.B, c.H, c.N) || !strides_ok(c.ks, c.B, c.Hk, c.N)) return TK_ATTN_ERR_UNSUPPORTED;
  if ((long long)c.B * c.N > 0x7fffffffLL ||
      (long long)c.B * c.N * ((long long)c.H + c.Hk) >= (1LL << 40))
    return TK_ATTN_ERR_UNSUPPORTED;
  return TK_ATTN_OK;
}

// Every range of `out` against every other and against the inputs.
int check_overlap(const uintptr_t *out, const size_t *out_n, int n_out, const uintptr_t *in,
                  const size_t *in_n, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = i + 1; j < n_out; ++j)
      if (ranges_overlap(out[i], out_n[i], out[j], out_n[j])) return TK_ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < n_in; ++j)
      if (ranges_overlap(out[i], out_n[i], in[j], in_n[j])) return TK_ATTN_ERR_INVALID_ARG;
  }
  return TK_ATTN_OK;
}

void fill(NrParams &p, const Call &c) {
  p.x[0] = {static_cast<const __nv_bfloat16 *>(c.q), c.qs[0], c.qs[1], c.qs[2]};
  p.x[1] = {static_cast<const __nv_bfloat16 *>(c.k), c.ks[0], c.ks[1], c.ks[2]};
  p.w[0] = c.qw;
  p.w[1] = c.kw;
  p.w_f32 = c.w_f32;
  p.turns = reinterpret_cast<const uint64_t *>(c.turns);
  p.pos = c.positions;
  p.eps = c.eps;
  p.B = c.B;
  p.N = c.N;
  p.H[0] = c.H;
  p.H[1] = c.Hk;
  p.rot = c.rot;
  p.dw_part = nullptr;
}

// Heads a row group takes for one token: fewer until there are blocks for
// every SM (each run of heads computes the token's sines and cosines again), and
// more again where the runs would pass the grid's second dimension.
void split(NrParams &p, int D, int threads, int most, int max_runs, long long blocks_wanted) {
  const int groups = threads / (D / 8);
  p.tiles = (int)(((long long)p.B * p.N + groups - 1) / groups);
  auto runs = [&](int hpg) {
    return ((long long)p.H[0] + hpg - 1) / hpg + ((long long)p.H[1] + hpg - 1) / hpg;
  };
  int hpg = most;
  while (hpg > 1 && p.tiles * runs(hpg) < blocks_wanted) hpg /= 2;
  while (runs(hpg) > max_runs) hpg *= 2;
  p.hpg = hpg;
  for (int i = 0; i < 2; ++i) p.chunks[i] = (p.H[i] + hpg - 1) / hpg;
}

template <bool kBwd>
cudaError_t launch(const NrParams &p, int D, bool halves, dim3 grid, cudaStream_t s) {
  const auto kernel = D == 64 ? (halves ? tk_norm_rope_kernel<64, true, kBwd>
                                        : tk_norm_rope_kernel<64, false, kBwd>)
                              : (halves ? tk_norm_rope_kernel<128, true, kBwd>
                                        : tk_norm_rope_kernel<128, false, kBwd>);
  return launch_overlapped(kernel, grid, kBwd ? kNrBwdThreads : kNrFwdThreads, 0, s, p);
}

}  // namespace
}  // namespace tkattn

using namespace tkattn;

extern "C" int tk_attn_qk_norm_rope_check_args(
    const void *q, const long long *q_strides, const void *k, const long long *k_strides,
    const void *q_weight, const void *k_weight, int weight_f32, const unsigned long long *turns,
    const int *positions, const void *q_out, const void *k_out, int B, int H, int Hk, int N, int D,
    int rot, int interleaved, float eps) {
  (void)interleaved;
  const Call c = {q, k, q_weight, k_weight, q_strides, k_strides, turns, positions,
                  B, H, Hk, N, D, rot, weight_f32, eps};
  if (!q_out || !k_out) return TK_ATTN_ERR_INVALID_ARG;
  int st = check_common(c);
  if (st) return st;
  if (((uintptr_t)q_out | (uintptr_t)k_out) & 15u) return TK_ATTN_ERR_UNSUPPORTED;
  const size_t wb = (size_t)D * (weight_f32 ? 4 : 2);
  const uintptr_t out[2] = {(uintptr_t)q_out, (uintptr_t)k_out};
  const size_t out_n[2] = {(size_t)B * H * N * D * 2, (size_t)B * Hk * N * D * 2};
  const uintptr_t in[6] = {(uintptr_t)q, (uintptr_t)k, (uintptr_t)q_weight, (uintptr_t)k_weight,
                           (uintptr_t)turns, (uintptr_t)positions};
  const size_t in_n[6] = {extent(q_strides, B, H, N, D), extent(k_strides, B, Hk, N, D), wb, wb,
                          (size_t)rot * 4, positions ? (size_t)B * N * 4 : 0};
  return check_overlap(out, out_n, 2, in, in_n, 6);
}

extern "C" int tk_attn_qk_norm_rope(
    const void *q, const long long *q_strides, const void *k, const long long *k_strides,
    const void *q_weight, const void *k_weight, int weight_f32, const unsigned long long *turns,
    const int *positions, void *q_out, void *k_out, int B, int H, int Hk, int N, int D, int rot,
    int interleaved, float eps, tk_attn_stream_t stream) {
  int st = tk_attn_qk_norm_rope_check_args(q, q_strides, k, k_strides, q_weight, k_weight,
                                           weight_f32, turns, positions, q_out, k_out, B, H, Hk, N,
                                           D, rot, interleaved, eps);
  if (st) return st;
  DeviceView dv;
  if ((st = device_view(&dv))) return st;
  const Call c = {q, k, q_weight, k_weight, q_strides, k_strides, turns, positions,
                  B, H, Hk, N, D, rot, weight_f32, eps};
  NrParams p;
  fill(p, c);
  void *const outs[2] = {q_out, k_out};
  for (int i = 0; i < 2; ++i) {
    p.y[i] = static_cast<__nv_bfloat16 *>(outs[i]);
    p.yn[i] = D;
    p.yh[i] = (long long)N * D;
    p.yb[i] = (long long)p.H[i] * N * D;
    p.dy[i] = {nullptr, 0, 0, 0};
  }
  split(p, D, kNrFwdThreads, kNrFwdHeads, 65535, 16LL * dv.num_sms);
  const dim3 grid(p.tiles, p.chunks[0] + p.chunks[1]);
  p.early = one_wave((long long)grid.x * grid.y, dv.num_sms);
  return launch<false>(p, D, !interleaved, grid, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? TK_ATTN_OK
             : TK_ATTN_ERR_LAUNCH;
}

extern "C" size_t tk_attn_qk_norm_rope_bwd_workspace_bytes(int D) {
  return D == 64 || D == 128 ? (size_t)kNrBwdMaxBlocks * D * sizeof(float) : 0;
}

extern "C" int tk_attn_qk_norm_rope_bwd_check_args(
    const void *q, const long long *q_strides, const void *k, const long long *k_strides,
    const void *q_weight, const void *k_weight, int weight_f32, const unsigned long long *turns,
    const int *positions, const void *dq_out, const long long *dq_out_strides, const void *dk_out,
    const long long *dk_out_strides, const void *dq, const long long *dq_strides, const void *dk,
    const long long *dk_strides, const float *dq_weight, const float *dk_weight, int B, int H,
    int Hk, int N, int D, int rot, int interleaved, float eps, const void *workspace,
    size_t workspace_bytes) {
  (void)interleaved;
  const Call c = {q, k, q_weight, k_weight, q_strides, k_strides, turns, positions,
                  B, H, Hk, N, D, rot, weight_f32, eps};
  if (!dq_out || !dk_out || !dq || !dk || !dq_weight || !dk_weight || !workspace ||
      !dq_out_strides || !dk_out_strides || !dq_strides || !dk_strides)
    return TK_ATTN_ERR_INVALID_ARG;
  int st = check_common(c);
  if (st) return st;
  if (((uintptr_t)dq_out | (uintptr_t)dk_out | (uintptr_t)dq | (uintptr_t)dk |
       (uintptr_t)workspace) & 15u ||
      ((uintptr_t)dq_weight | (uintptr_t)dk_weight) & 3u)
    return TK_ATTN_ERR_UNSUPPORTED;
  if (!strides_ok(dq_out_strides, B, H, N) || !strides_ok(dk_out_strides, B, Hk, N) ||
      !strides_ok(dq_strides, B, H, N) || !strides_ok(dk_strides, B, Hk, N))
    return TK_ATTN_ERR_UNSUPPORTED;
  if (!distinct(dq_strides, B, H, N, D) || !distinct(dk_strides, B, Hk, N, D))
    return TK_ATTN_ERR_INVALID_ARG;
  const size_t need = tk_attn_qk_norm_rope_bwd_workspace_bytes(D);
  if (workspace_bytes < need) return TK_ATTN_ERR_INVALID_ARG;
  const size_t wb = (size_t)D * (weight_f32 ? 4 : 2);
  const uintptr_t out[5] = {(uintptr_t)dq, (uintptr_t)dk, (uintptr_t)dq_weight,
                            (uintptr_t)dk_weight, (uintptr_t)workspace};
  const size_t out_n[5] = {extent(dq_strides, B, H, N, D), extent(dk_strides, B, Hk, N, D),
                           (size_t)D * 4, (size_t)D * 4, need};
  const uintptr_t in[8] = {(uintptr_t)q, (uintptr_t)k, (uintptr_t)q_weight, (uintptr_t)k_weight,
                           (uintptr_t)turns, (uintptr_t)positions, (uintptr_t)dq_out,
                           (uintptr_t)dk_out};
  const size_t in_n[8] = {extent(q_strides, B, H, N, D), extent(k_strides, B, Hk, N, D), wb, wb,
                          (size_t)rot * 4, positions ? (size_t)B * N * 4 : 0,
                          extent(dq_out_strides, B, H, N, D), extent(dk_out_strides, B, Hk, N, D)};
  // dq and dk may lie in one fused gradient, a token's query and key heads in
  // turn: their extents then overlap, their elements do not.
  for (int i = 0; i < 5; ++i) {
    for (int j = i + 1; j < 5; ++j) {
      if (i == 0 && j == 1 &&
          interleave_apart(out[0], dq_strides, H, out[1], dk_strides, Hk, B, N, D))
        continue;
      if (ranges_overlap(out[i], out_n[i], out[j], out_n[j])) return TK_ATTN_ERR_INVALID_ARG;
    }
    for (int j = 0; j < 8; ++j)
      if (ranges_overlap(out[i], out_n[i], in[j], in_n[j])) return TK_ATTN_ERR_INVALID_ARG;
  }
  return TK_ATTN_OK;
}

extern "C" int tk_attn_qk_norm_rope_bwd(
    const void *q, const long long *q_strides, const void *k, const long long *k_strides,
    const void *q_weight, const void *k_weight, int weight_f32, const unsigned long long *turns,
    const int *positions, const void *dq_out, const long long *dq_out_strides, const void *dk_out,
    const long long *dk_out_strides, void *dq, const long long *dq_strides, void *dk,
    const long long *dk_strides, float *dq_weight, float *dk_weight, int B, int H, int Hk, int N,
    int D, int rot, int interleaved, float eps, void *workspace, size_t workspace_bytes,
    tk_attn_stream_t stream) {
  int st = tk_attn_qk_norm_rope_bwd_check_args(
      q, q_strides, k, k_strides, q_weight, k_weight, weight_f32, turns, positions, dq_out,
      dq_out_strides, dk_out, dk_out_strides, dq, dq_strides, dk, dk_strides, dq_weight, dk_weight,
      B, H, Hk, N, D, rot, interleaved, eps, workspace, workspace_bytes);
  if (st) return st;
  DeviceView dv;
  if ((st = device_view(&dv))) return st;
  const Call c = {q, k, q_weight, k_weight, q_strides, k_strides, turns, positions,
                  B, H, Hk, N, D, rot, weight_f32, eps};
  NrParams p;
  fill(p, c);
  p.y[0] = static_cast<__nv_bfloat16 *>(dq);
  p.y[1] = static_cast<__nv_bfloat16 *>(dk);
  const long long *const ys[2] = {dq_strides, dk_strides};
  for (int i = 0; i < 2; ++i) {
    p.yb[i] = ys[i][0];
    p.yh[i] = ys[i][1];
    p.yn[i] = ys[i][2];
  }
  p.dy[0] = {static_cast<const __nv_bfloat16 *>(dq_out), dq_out_strides[0], dq_out_strides[1],
             dq_out_strides[2]};
  p.dy[1] = {static_cast<const __nv_bfloat16 *>(dk_out), dk_out_strides[0], dk_out_strides[1],
             dk_out_strides[2]};
  // As many blocks as are resident at once, each over several tiles.
  const int blocks = kNrBwdBlocks * dv.num_sms;
  split(p, D, kNrBwdThreads, kNrBwdHeads, kNrBwdMaxBlocks, blocks);
  p.dw_part = static_cast<float *>(workspace);
  p.early = 1;
  const int runs = p.chunks[0] + p.chunks[1];
  int cols = blocks / runs;
  cols = cols < 1 ? 1 : cols > p.tiles ? p.tiles : cols;
  if ((long long)cols * runs > kNrBwdMaxBlocks) cols = kNrBwdMaxBlocks / runs;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (launch<true>(p, D, !interleaved, dim3(cols, runs), s) != cudaSuccess)
    return TK_ATTN_ERR_LAUNCH;
  return launch_overlapped(tk_norm_rope_dw_kernel, dim3(D / 32, 2), 1024, 0, s, p.dw_part,
                           cols * p.chunks[0], cols * p.chunks[1], D, dq_weight,
                           dk_weight) == cudaSuccess
             ? TK_ATTN_OK
             : TK_ATTN_ERR_LAUNCH;
}
