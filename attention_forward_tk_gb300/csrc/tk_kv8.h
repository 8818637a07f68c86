// tk_kv8.h -- the 8-bit paged cache's index arithmetic, for the kernels and
// (compiled as plain C++) for checks on the CPU.
//
// A cache holds k and v payloads [num_pages, Hkv, page, D] in E4M3 and int8
// exponents [num_pages, Hkv]; the value held is payload * 2^exponent.  A
// sequence's position t lies in row t % page of page table[b][t / page].
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define TK_HD __host__ __device__ __forceinline__
#else
#define TK_HD inline
#endif

namespace tkattn {

// Exponents a write gives: E4M3's least subnormal 2^-9 times 2^-117 is bf16's
// least normal, and 448 * 2^119 is below bf16's largest value, so every value
// held is a bf16 value.
constexpr int kKv8ExpMin = -117, kKv8ExpMax = 119;

struct Kv8Geom {
  int num_pages, Hkv, page, D;
  int max_pages;     // entries of a sequence's page table
  int table_stride;  // entries from one sequence's table to the next
};

// Positions a page table can hold.
TK_HD long long kv8_capacity(const Kv8Geom &g) { return (long long)g.max_pages * g.page; }

TK_HD bool kv8_page_ok(const Kv8Geom &g, int id) { return id >= 0 && id < g.num_pages; }

// Byte (= element) offset of row `row` of head h in page id.
TK_HD long long kv8_row_offset(const Kv8Geom &g, int id, int h, int row) {
  return (((long long)id * g.Hkv + h) * g.page + row) * g.D;
}

TK_HD long long kv8_exp_offset(const Kv8Geom &g, int id, int h) {
  return (long long)id * g.Hkv + h;
}

TK_HD long long kv8_table_offset(const Kv8Geom &g, int b, int slot) {
  return (long long)b * g.table_stride + slot;
}

// A sequence's length as the kernels use it: within [0, capacity].  `bad` is
// set when it was not.
TK_HD int kv8_length(const Kv8Geom &g, int len, bool *bad) {
  const long long cap = kv8_capacity(g);
  if (len < 0) {
    *bad = true;
    return 0;
  }
  if ((long long)len > cap) {
    *bad = true;
    return (int)cap;
  }
  return len;
}

// A write's rows [0, n) at positions [start, start + n): the rows that lie
// inside the table.  None when start is outside it.
TK_HD int kv8_write_rows(const Kv8Geom &g, int start, int count, int N, bool *bad) {
  const long long cap = kv8_capacity(g);
  int n = count;
  if (n < 0 || n > N) {
    *bad = true;
    n = n < 0 ? 0 : N;
  }
  if (n == 0) return 0;
  if (start < 0 || (long long)start >= cap) {
    *bad = true;
    return 0;
  }
  if ((long long)start + n > cap) {
    *bad = true;
    n = (int)(cap - start);
  }
  return n;
}

// Pages that N rows can touch, wherever they start.
TK_HD int kv8_span(int N, int page) { return (int)(((long long)N + page - 2) / page + 1); }

// The least exponent e in [kKv8ExpMin, kKv8ExpMax] with 448 * 2^e >= m, for a
// finite magnitude given as the bits of a bf16 value (sign clear).
TK_HD int kv8_exponent(uint32_t bits) {
  const int x = (int)(bits >> 7) - 127;  // floor(log2) of a normal value
  const int e = x - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0);  // 448 = 1.75 * 2^8
  return e < kKv8ExpMin ? kKv8ExpMin : e > kKv8ExpMax ? kKv8ExpMax : e;
}

}  // namespace tkattn
