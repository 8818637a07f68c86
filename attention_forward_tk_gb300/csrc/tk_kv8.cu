// tk_kv8.cu -- host side of the 8-bit paged cache: argument checks and
// launches of the write, the read-back and the attention over it (the C ABI is
// in tk_attn.h; the kernels in tk_kv8_copy.cuh, tk_kv8_decode.cuh and
// tk_kv8_chunk.cuh).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "tk_attn.h"
#include "tk_device.h"
#include "tk_kv8.h"
#include "tk_kv8_chunk.cuh"
#include "tk_kv8_copy.cuh"
#include "tk_kv8_decode.cuh"

namespace tkattn {
namespace {

// Kernel attributes, once per device.
struct Kv8Device {
  std::once_flag once;
  bool ok = false;
};
Kv8Device g_kv8_dev[kMaxDevices];

template <int D, int kNT>
bool configure_decode() {
  return cudaFuncSetAttribute(tk_kv8_decode_kernel<D, kNT>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              DecCfg<D, kNT>::kSmem) == cudaSuccess;
}

template <int D, bool kPair>
bool configure_chunk() {
  if (cudaFuncSetAttribute(tk_kv8_chunk_kernel<D, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           ChunkCfg<D>::kSmemAlloc) != cudaSuccess)
    return false;
  // the register split between warpgroups assumes exactly 128 a thread at launch
  cudaFuncAttributes fa;
  return cudaFuncGetAttributes(&fa, tk_kv8_chunk_kernel<D, kPair>) == cudaSuccess && fa.numRegs == 128;
}

int kv8_device(DeviceView *dv) {
  const int st = device_view(dv);
  if (st) return st;
  Kv8Device &d = g_kv8_dev[dv->index];
  std::call_once(d.once, [&d] {
    d.ok = configure_decode<64, 1>() && configure_decode<64, 2>() && configure_decode<64, 3>() &&
           configure_decode<64, 4>() && configure_decode<64, 5>() && configure_decode<128, 1>() &&
           configure_decode<128, 2>() && configure_decode<128, 3>() &&
           configure_chunk<64, false>() && configure_chunk<64, true>() &&
           configure_chunk<128, false>();
  });
  return d.ok ? TK_ATTN_OK : TK_ATTN_ERR_LAUNCH;
}

int check_geom(const void *k_cache, const void *v_cache, const void *k_exp, const void *v_exp,
               const int *table, int num_pages, int Hkv, int page, int D, int max_pages,
               int table_stride) {
  if (!k_cache || !v_cache || !k_exp || !v_exp || !table) return TK_ATTN_ERR_INVALID_ARG;
  if (num_pages <= 0 || Hkv <= 0 || max_pages <= 0 || table_stride < max_pages)
    return TK_ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return TK_ATTN_ERR_UNSUPPORTED;
  if (page != 16 && page != 32 && page != 64 && page != 128) return TK_ATTN_ERR_UNSUPPORTED;
  if (((uintptr_t)k_cache | (uintptr_t)v_cache) & 15u || (uintptr_t)table & 3u)
    return TK_ATTN_ERR_UNSUPPORTED;
  // (positions are rounded up to whole tiles in 32 bits)
  if ((long long)max_pages * page > 0x7fffff00LL || 2LL * Hkv > 65535 ||
      (long long)num_pages * Hkv * page > 0x7fffffffLL)
    return TK_ATTN_ERR_UNSUPPORTED;
  return TK_ATTN_OK;
}

Kv8Geom geom(int num_pages, int Hkv, int page, int D, int max_pages, int table_stride) {
  return Kv8Geom{num_pages, Hkv, page, D, max_pages, table_stride};
}

struct Range {
  const void *p;
  size_t n;
};

// No written range may share a byte with another or with one that is read.
int check_ranges(const Range *out, int n_out, const Range *in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = i + 1; j < n_out; ++j)
      if (ranges_overlap((uintptr_t)out[i].p, out[i].n, (uintptr_t)out[j].p, out[j].n))
        return TK_ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < n_in; ++j)
      if (ranges_overlap((uintptr_t)out[i].p, out[i].n, (uintptr_t)in[j].p, in[j].n))
        return TK_ATTN_ERR_INVALID_ARG;
  }
  return TK_ATTN_OK;
}

int log2i(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

// (a thread's registers hold its part of a whole page)
template <int kPage>
cudaError_t launch_write(const Kv8WriteParams &p, int D, dim3 grid, cudaStream_t s) {
  return launch_overlapped(
      D == 64 ? tk_kv8_write_kernel<64, kPage> : tk_kv8_write_kernel<128, kPage>, grid,
      kKv8Threads, 0, s, p);
}

size_t table_bytes(int B, int max_pages, int table_stride) {
  return ((size_t)(B - 1) * table_stride + max_pages) * 4;
}

}  // namespace
}  // namespace tkattn

using namespace tkattn;

extern "C" int tk_attn_kv8_write_check_args(
    const void *k, const long long *k_strides, const void *v, const long long *v_strides,
    const void *k_cache, const void *v_cache, const void *k_exp, const void *v_exp,
    const int *page_table, const int *start, const int *counts, int B, int Hkv, int N, int D,
    int num_pages, int page, int max_pages, int table_stride) {
  if (!k || !v || !k_strides || !v_strides || !start) return TK_ATTN_ERR_INVALID_ARG;
  if (B <= 0 || N <= 0) return TK_ATTN_ERR_INVALID_ARG;
  const int st = check_geom(k_cache, v_cache, k_exp, v_exp, page_table, num_pages, Hkv, page, D,
                            max_pages, table_stride);
  if (st) return st;
  if (((uintptr_t)k | (uintptr_t)v) & 15u || ((uintptr_t)start | (uintptr_t)counts) & 3u)
    return TK_ATTN_ERR_UNSUPPORTED;
  const int dims[3] = {B, Hkv, N};  // (the stride of a dimension of one says nothing)
  for (const long long *s : {k_strides, v_strides})
    for (int i = 0; i < 3; ++i)
      if (dims[i] > 1 && (s[i] < 0 || s[i] % 8 || s[i] >= (1LL << 40))) return TK_ATTN_ERR_UNSUPPORTED;
  if (B > 65535) return TK_ATTN_ERR_UNSUPPORTED;
  const size_t payload = (size_t)num_pages * Hkv * page * D, exps = (size_t)num_pages * Hkv;
  auto extent = [&](const long long *s) {
    return 2 * (size_t)((B - 1) * s[0] + (Hkv - 1) * s[1] + (N - 1) * s[2] + D);
  };
  const Range out[4] = {{k_cache, payload}, {v_cache, payload}, {k_exp, exps}, {v_exp, exps}};
  const Range in[5] = {{k, extent(k_strides)},
                       {v, extent(v_strides)},
                       {page_table, table_bytes(B, max_pages, table_stride)},
                       {start, (size_t)B * 4},
                       {counts, counts ? (size_t)B * 4 : 0}};
  return check_ranges(out, 4, in, 5);
}

extern "C" int tk_attn_kv8_write(const void *k, const long long *k_strides, const void *v,
                                 const long long *v_strides, void *k_cache, void *v_cache,
                                 void *k_exp, void *v_exp, const int *page_table, const int *start,
                                 const int *counts, int B, int Hkv, int N, int D, int num_pages,
                                 int page, int max_pages, int table_stride,
                                 tk_attn_stream_t stream) {
  int st = tk_attn_kv8_write_check_args(k, k_strides, v, v_strides, k_cache, v_cache, k_exp, v_exp,
                                        page_table, start, counts, B, Hkv, N, D, num_pages, page,
                                        max_pages, table_stride);
  if (st) return st;
  DeviceView dv;
  if ((st = kv8_device(&dv))) return st;
  Kv8WriteParams p;
  p.g = geom(num_pages, Hkv, page, D, max_pages, table_stride);
  const void *const src[2] = {k, v};
  const long long *const ss[2] = {k_strides, v_strides};
  void *const pay[2] = {k_cache, v_cache}, *const ex[2] = {k_exp, v_exp};
  for (int i = 0; i < 2; ++i) {
    p.src[i] = static_cast<const __nv_bfloat16 *>(src[i]);
    p.sb[i] = ss[i][0];
    p.sh[i] = ss[i][1];
    p.sn[i] = ss[i][2];
    p.payload[i] = static_cast<uint8_t *>(pay[i]);
    p.exps[i] = static_cast<int8_t *>(ex[i]);
  }
  p.table = page_table;
  p.start = start;
  p.counts = counts;
  p.B = B;
  p.N = N;
  p.err = dv.err_word;
  const dim3 grid(kv8_span(N, page), 2 * Hkv, B);
  p.early = one_wave((long long)grid.x * grid.y * grid.z, dv.num_sms);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = page == 16   ? launch_write<16>(p, D, grid, s)
                        : page == 32 ? launch_write<32>(p, D, grid, s)
                        : page == 64 ? launch_write<64>(p, D, grid, s)
                                     : launch_write<128>(p, D, grid, s);
  return e == cudaSuccess ? TK_ATTN_OK : TK_ATTN_ERR_LAUNCH;
}

extern "C" int tk_attn_kv8_read_check_args(const void *k_cache, const void *v_cache,
                                           const void *k_exp, const void *v_exp,
                                           const int *page_table, const int *lengths,
                                           const void *k, const void *v, int B, int Hkv, int N,
                                           int D, int num_pages, int page, int max_pages,
                                           int table_stride) {
  if (!lengths || !k || !v || B <= 0 || N <= 0) return TK_ATTN_ERR_INVALID_ARG;
  const int st = check_geom(k_cache, v_cache, k_exp, v_exp, page_table, num_pages, Hkv, page, D,
                            max_pages, table_stride);
  if (st) return st;
  if (((uintptr_t)k | (uintptr_t)v) & 15u || (uintptr_t)lengths & 3u)
    return TK_ATTN_ERR_UNSUPPORTED;
  if (B > 65535) return TK_ATTN_ERR_UNSUPPORTED;
  const size_t payload = (size_t)num_pages * Hkv * page * D, exps = (size_t)num_pages * Hkv;
  const size_t dense = (size_t)B * Hkv * N * D * 2;
  const Range out[2] = {{k, dense}, {v, dense}};
  const Range in[6] = {{k_cache, payload},
                       {v_cache, payload},
                       {k_exp, exps},
                       {v_exp, exps},
                       {page_table, table_bytes(B, max_pages, table_stride)},
                       {lengths, (size_t)B * 4}};
  return check_ranges(out, 2, in, 6);
}

extern "C" int tk_attn_kv8_read(const void *k_cache, const void *v_cache, const void *k_exp,
                                const void *v_exp, const int *page_table, const int *lengths,
                                void *k, void *v, int B, int Hkv, int N, int D, int num_pages,
                                int page, int max_pages, int table_stride,
                                tk_attn_stream_t stream) {
  int st = tk_attn_kv8_read_check_args(k_cache, v_cache, k_exp, v_exp, page_table, lengths, k, v,
                                       B, Hkv, N, D, num_pages, page, max_pages, table_stride);
  if (st) return st;
  DeviceView dv;
  if ((st = kv8_device(&dv))) return st;
  Kv8ReadParams p;
  p.g = geom(num_pages, Hkv, page, D, max_pages, table_stride);
  p.payload[0] = static_cast<const uint8_t *>(k_cache);
  p.payload[1] = static_cast<const uint8_t *>(v_cache);
  p.exps[0] = static_cast<const int8_t *>(k_exp);
  p.exps[1] = static_cast<const int8_t *>(v_exp);
  p.table = page_table;
  p.lengths = lengths;
  p.dst[0] = static_cast<__nv_bfloat16 *>(k);
  p.dst[1] = static_cast<__nv_bfloat16 *>(v);
  p.B = B;
  p.N = N;
  p.err = dv.err_word;
  const dim3 grid((int)(((long long)N + 63) / 64), 2 * Hkv, B);
  p.early = one_wave((long long)grid.x * grid.y * grid.z, dv.num_sms);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      launch_overlapped(D == 64 ? tk_kv8_read_kernel<64> : tk_kv8_read_kernel<128>, grid,
                        kKv8Threads, 0, s, p);
  return e == cudaSuccess ? TK_ATTN_OK : TK_ATTN_ERR_LAUNCH;
}

namespace tkattn {
namespace {

// Tiles of eight query rows that a warp of the streaming kernel holds for a
// call's Nq * G rows, or 0 where the rows go to the 128-row tiles of the tensor
// core: past 24 rows at D = 128 and 40 at D = 64 the registers spill.  (32 sequences
// of up to 32768 positions, 2 key heads of 64: 8 to 40 rows in steps of 8 take 33, 43, 50,
// 68 and 82 us, 48 and 64 rows on the tensor core 90 and 92.)
int row_tiles(int G, int Nq, int D) {
  const long long tiles = ((long long)Nq * G + 7) / 8;
  return tiles <= (D == 64 ? 5 : 3) ? (int)tiles : 0;
}
// Runs the work is cut into: the CTAs that fit on the device at once.
int run_count(const DeviceView &dv, int tiles, int D) {
  if (tiles == 0) return dv.num_sms;
  const int per_sm = D == 64 ? (tiles <= 1   ? DecCfg<64, 1>::kCtasPerSm
                               : tiles <= 3 ? DecCfg<64, 3>::kCtasPerSm
                                            : DecCfg<64, 5>::kCtasPerSm)
                             : (tiles == 1 ? DecCfg<128, 1>::kCtasPerSm
                                           : DecCfg<128, 3>::kCtasPerSm);
  return per_sm * dv.num_sms;
}

bool sizes_ok(int B, int H, int Hkv, int Nq, int D) {
  return B > 0 && H > 0 && Hkv > 0 && Nq > 0 && H % Hkv == 0 && (D == 64 || D == 128);
}

size_t prefix_bytes(int B) { return ((size_t)B * 8 + 8 + 15) / 16 * 16; }

size_t workspace_for(const DeviceView &dv, int B, int G, int Nq, int D) {
  const int tiles = row_tiles(G, Nq, D);
  const int rows = tiles ? 8 * tiles : kChunkRows;
  return prefix_bytes(B) + (size_t)run_count(dv, tiles, D) * 2 * rows * (D + 4) * sizeof(float);
}

template <int D, int kNT>
cudaError_t launch_decode(const Kv8AttnParams &p, cudaStream_t s) {
  const cudaError_t e = launch_overlapped(tk_kv8_decode_kernel<D, kNT>, p.ctas, kDecThreads,
                                          DecCfg<D, kNT>::kSmem, s, p);
  if (e != cudaSuccess) return e;
  const int rows = p.Nq * p.G;
  // A warp a row where there are more than two rows a run: 64 sequences of up to
  // 2048 positions (2048 rows, D = 128) 40.2 -> 36.9 us, 16 of up to 16384 with five
  // drafts (1280 rows, D = 64) 35.0 -> 33.7 us; with 512 rows, of 14 partials each,
  // a block a row is the faster, 18.8 us against 20.4.
  if ((long long)p.B * p.g.Hkv * rows > 2LL * p.ctas)
    return launch_overlapped(tk_kv8_merge_kernel<D, true>,
                             dim3(p.g.Hkv, p.B, (rows + kMergeWarps - 1) / kMergeWarps),
                             kMergeWarps * 32, 0, s, p);
  return launch_overlapped(tk_kv8_merge_kernel<D, false>, dim3(p.g.Hkv, p.B, rows),
                           kMergeWarps * 32, 0, s, p);
}

template <int D>
cudaError_t launch_chunk(const Kv8AttnParams &p, cudaStream_t s) {
  const long long rows = (long long)p.g.num_pages * p.g.Hkv * p.g.page;
  CUtensorMap tk, tv;
  if (!make_map_bytes(&tk, p.k, rows, D, p.g.page) || !make_map_bytes(&tv, p.v, rows, D, p.g.page))
    return cudaErrorInvalidValue;
  const cudaError_t e =
      launch_overlapped(D == 64 && p.pair ? tk_kv8_chunk_kernel<D, D == 64>
                                          : tk_kv8_chunk_kernel<D, false>,
                        p.ctas, kChunkThreads, ChunkCfg<D>::kSmemAlloc, s, tk, tv, p);
  if (e != cudaSuccess) return e;
  // Four runs a unit or more on average: the partials of a row are the parallel
  // work; else the rows are.
  const long long units = (long long)p.B * p.g.Hkv * (((long long)p.Nq * p.G + 255) / 256);
  if (4 * units <= p.ctas)
    return launch_overlapped(tk_kv8_chunk_merge_deep_kernel<D>,
                             dim3((unsigned)(p.Nq * p.G), p.g.Hkv, p.B), kMergeWarps * 32, 0, s, p);
  return launch_overlapped(tk_kv8_chunk_merge_kernel<D>,
                           dim3((unsigned)(((long long)p.Nq * p.G + 31) / 32), p.g.Hkv, p.B), 256, 0,
                           s, p);
}

}  // namespace
}  // namespace tkattn

extern "C" size_t tk_attn_fwd_kv8_workspace_bytes(int B, int H, int Hkv, int Nq, int D) {
  DeviceView dv;
  if (!sizes_ok(B, H, Hkv, Nq, D) || device_view(&dv)) return 0;
  return workspace_for(dv, B, H / Hkv, Nq, D);
}

extern "C" int tk_attn_fwd_kv8_check_args(const void *q, const void *k_cache, const void *v_cache,
                                          const void *k_exp, const void *v_exp,
                                          const int *page_table, const int *lengths,
                                          const int *counts, const void *o, const float *lse,
                                          int B, int H, int Hkv, int Nq, int D, int num_pages,
                                          int page, int max_pages, int table_stride, float scale,
                                          int causal, const void *workspace,
                                          size_t workspace_bytes) {
  (void)causal;
  if (!q || !lengths || !o || !lse || !workspace) return TK_ATTN_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || Nq <= 0 || Hkv <= 0 || H % Hkv) return TK_ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return TK_ATTN_ERR_INVALID_ARG;
  const int st = check_geom(k_cache, v_cache, k_exp, v_exp, page_table, num_pages, Hkv, page, D,
                            max_pages, table_stride);
  if (st) return st;
  if (((uintptr_t)q | (uintptr_t)o | (uintptr_t)lse | (uintptr_t)workspace) & 15u ||
      ((uintptr_t)lengths | (uintptr_t)counts) & 3u)
    return TK_ATTN_ERR_UNSUPPORTED;
  const long long G = H / Hkv;
  if (B > 65535 || Nq * G * G > 0x7fffffffLL ||
      (long long)Hkv * (((long long)Nq * G + 7) / 8) > 0x7fffffffLL ||
      (long long)B * H > 0x7fffffffLL)
    return TK_ATTN_ERR_UNSUPPORTED;
  // few rows count units of 64 positions in 32 bits (with room for a share)
  if ((long long)B * Hkv * ((long long)max_pages * page / 64 + 1) > (1LL << 30))
    return TK_ATTN_ERR_UNSUPPORTED;
  const size_t payload = (size_t)num_pages * Hkv * page * D, exps = (size_t)num_pages * Hkv;
  const size_t dense = (size_t)B * H * Nq * D * 2;
  const Range out[3] = {{o, dense}, {lse, (size_t)B * H * Nq * 4}, {workspace, workspace_bytes}};
  const Range in[8] = {{q, dense},
                       {k_cache, payload},
                       {v_cache, payload},
                       {k_exp, exps},
                       {v_exp, exps},
                       {page_table, table_bytes(B, max_pages, table_stride)},
                       {lengths, (size_t)B * 4},
                       {counts, counts ? (size_t)B * 4 : 0}};
  return check_ranges(out, 3, in, 8);
}

extern "C" int tk_attn_fwd_kv8(const void *q, const void *k_cache, const void *v_cache,
                               const void *k_exp, const void *v_exp, const int *page_table,
                               const int *lengths, const int *counts, void *o, float *lse, int B,
                               int H, int Hkv, int Nq, int D, int num_pages, int page,
                               int max_pages, int table_stride, float scale, int causal,
                               void *workspace, size_t workspace_bytes, tk_attn_stream_t stream) {
  int st = tk_attn_fwd_kv8_check_args(q, k_cache, v_cache, k_exp, v_exp, page_table, lengths,
                                      counts, o, lse, B, H, Hkv, Nq, D, num_pages, page, max_pages,
                                      table_stride, scale, causal, workspace, workspace_bytes);
  if (st) return st;
  DeviceView dv;
  if ((st = kv8_device(&dv))) return st;
  if (workspace_bytes < workspace_for(dv, B, H / Hkv, Nq, D)) return TK_ATTN_ERR_INVALID_ARG;
  Kv8AttnParams p;
  p.g = geom(num_pages, Hkv, page, D, max_pages, table_stride);
  p.page_log2 = log2i(page);
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.k = static_cast<const uint8_t *>(k_cache);
  p.v = static_cast<const uint8_t *>(v_cache);
  p.ke = static_cast<const int8_t *>(k_exp);
  p.ve = static_cast<const int8_t *>(v_exp);
  p.table = page_table;
  p.lengths = lengths;
  p.counts = counts;
  p.o = static_cast<__nv_bfloat16 *>(o);
  p.lse = lse;
  p.B = B;
  p.H = H;
  p.G = H / Hkv;
  p.g_mul = p.G == 1 ? 0u : (unsigned)((1ull << 32) / p.G + 1);
  p.Nq = Nq;
  p.causal = causal != 0;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  const int tiles = row_tiles(p.G, Nq, D);
  p.tile_rows = 8 * tiles;
  // Both tiles on the same rows where those fill one: 110 -> 90 us at D = 64 (32
  // sequences of up to 32768 positions, 48 rows a head); at D = 128, where a value
  // tile takes twice the conversion, 139 -> 148 us.
  p.pair = D == 64 && (long long)Nq * p.G <= 128;
  p.ctas = run_count(dv, tiles, D);
  p.err = dv.err_word;
  p.prefix = static_cast<long long *>(workspace);
  p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + prefix_bytes(B));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (D == 64) {
    switch (tiles) {
      case 0: e = launch_chunk<64>(p, s); break;
      case 1: e = launch_decode<64, 1>(p, s); break;
      case 2: e = launch_decode<64, 2>(p, s); break;
      case 3: e = launch_decode<64, 3>(p, s); break;
      case 4: e = launch_decode<64, 4>(p, s); break;
      default: e = launch_decode<64, 5>(p, s); break;
    }
  } else {
    switch (tiles) {
      case 0: e = launch_chunk<128>(p, s); break;
      case 1: e = launch_decode<128, 1>(p, s); break;
      case 2: e = launch_decode<128, 2>(p, s); break;
      default: e = launch_decode<128, 3>(p, s); break;
    }
  }
  return e == cudaSuccess ? TK_ATTN_OK : TK_ATTN_ERR_LAUNCH;
}
