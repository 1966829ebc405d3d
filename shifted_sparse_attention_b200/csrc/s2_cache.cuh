// s2_cache.cuh -- the paged cache of keys and values as the kernels see it:
// addresses of its rows, the batch's sequences, and the 4-bit row format.
//
// A page holds S rows (S = 16, 32, 64 or 128) of every key/value head, head
// by head: row (page, h, slot) starts at ((page·Hkv + h)·S + slot)·rowbytes, so
// the rows that one attention unit streams, a head's S rows of a page, are
// contiguous (4 KB and more in bf16).  All row numbers are 64-bit.
//
// 4-bit rows: byte j holds the code of channel j in its low half and that of
// channel j + D/2 in its high half; a row stands for min + scale·code, scale
// and min in bf16 ([.., 2] beside the codes).  The pairing of j with j + D/2
// is the rotation's, and lets a kernel split a 32-bit word into bf16 pairs
// with one shift and one mask per pair.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace s2 {

// Status flag: a page number, length or start of a batch was out of range.
constexpr int kCacheFlag = 0x2000;

struct CacheArgs {
  void* k;         // bf16 rows, or 4-bit codes
  void* v;
  void* k_scale;   // (scale, min) pairs, 4-bit caches only
  void* v_scale;
  const int* table;   // [B, width] page numbers
  const int* lens;    // [B] tokens of each sequence, the new ones included
  const int* starts;  // [B + 1] packed starts of the new tokens, or null: one per sequence
  long long pages;
  int heads;   // key/value heads
  int log2s;   // log2 of the rows of a page
  int B, T, width;
  int* status;
};

// Sequence b's new tokens are [first, first + n) of the packed axis; it has
// len tokens, the new ones included, so new token i is at place len - n + i.
struct Seq {
  int first, n, len;
};

// A sequence whose numbers are out of range is reported and left out (n = 0).
__device__ __forceinline__ Seq load_seq(const CacheArgs& c, int b) {
  Seq s;
  const int lo = c.starts ? c.starts[b] : b;
  const int hi = c.starts ? c.starts[b + 1] : b + 1;
  s.len = c.lens[b];
  s.first = lo;
  s.n = hi - lo;
  if (lo < 0 || hi < lo || hi > c.T || s.len < 0 || (long long)s.len > ((long long)c.width << c.log2s)) {
    atomicOr(c.status, kCacheFlag);
    s.n = 0;
    s.len = 0;
  }
  return s;
}

// Page that holds place p of sequence b; an entry that names no page is reported and reads page 0.
__device__ __forceinline__ int page_of(const CacheArgs& c, int b, int p) {
  int page = c.table[(size_t)b * c.width + (p >> c.log2s)];
  if ((unsigned)page >= (unsigned long long)c.pages) {
    atomicOr(c.status, kCacheFlag);
    page = 0;
  }
  return page;
}

// Number of the row of head h at place p on `page`.
__device__ __forceinline__ size_t row_of(const CacheArgs& c, int page, int h, int p) {
  return (((size_t)page * c.heads + h) << c.log2s) + (p & ((1 << c.log2s) - 1));
}

// (scale, min) of a 4-bit row as floats, from its packed bf16 pair.
__device__ __forceinline__ float2 q4_pair(uint32_t raw) {
  return make_float2(__uint_as_float(raw << 16), __uint_as_float(raw & 0xffff0000u));
}

}  // namespace s2
