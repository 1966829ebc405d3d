// s2_cache.cuh -- the paged cache of keys and values as the kernels see it:
// addresses of its rows, the batch's sequences, and the 4-bit row format.
//
// A page holds S rows (S = 16, 32, 64 or 128) of every key/value head, head
// by head: row (page, h, slot) starts at ((page·Hkv + h)·S + slot)·rowbytes, so
// the rows that one attention unit streams, a head's S rows of a page, are
// contiguous (4 KB and more in bf16).  Rows are fewer than 2^32; offsets are
// 64-bit.
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

// A sequence whose numbers are out of range is reported and left out (n = 0).  One without new tokens takes no part, and
// its length may be anything.
__device__ __forceinline__ Seq load_seq(const CacheArgs& c, int b) {
  Seq s;
  const int lo = c.starts ? c.starts[b] : b;
  const int hi = c.starts ? c.starts[b + 1] : b + 1;
  s.len = c.lens[b];
  s.first = lo;
  s.n = hi - lo;
  // (no short circuits: the length is asked for along with the starts, not after them)
  const bool beyond = (s.len < 0) | ((long long)s.len > ((long long)c.width << c.log2s));
  const bool bad = (lo < 0) | (hi < lo) | (hi > c.T) | ((hi > lo) & beyond);
  if (bad) atomicOr(c.status, kCacheFlag);
  if (bad | (hi == lo)) s.n = s.len = 0;
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

// A key's part in a score, s·(q·(128 + c)) + (m - 128 s)·sum(q), goes through numbers that are up to 19 times the largest
// of the row, so for a row near the end of 32 bits they would leave it.  The kernels work on 2^-5 of the score instead
// (exact: only powers of two), which scale_log2 makes up for:
//   (2^-5 s)·(q·(128 + c)) + (2^-12 m - 2^-5 s)·(128 sum(q)).
constexpr float kQ4ScoreUnit = 32.f, kQ4Bias = 128.f;
// {2^-5 s, 2^-12 m - 2^-5 s} of a key's (s, m).
__device__ __forceinline__ float2 q4_key(float2 pair) {
  const float s = pair.x * (1.f / kQ4ScoreUnit);
  return make_float2(s, fmaf(pair.y, 1.f / (kQ4ScoreUnit * kQ4Bias), -s));
}

// ---------------------------------------------------------------- cutting the work into equal pieces
// All sequences' work, weighed by `weight(b)`, forms one line that is cut into
// equal pieces, one per CTA.  The lengths are only known on the device, so
// every CTA adds the weights up by itself: they are a few KB, and in L2.
struct Line {
  long long total, piece;
};

// a / b of numbers >= 0: in 32 bits where they fit, which is a fraction of the time.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Shared memory of the two calls below: kThreads / 32 + 2 values.
template <int kThreads, typename Weight>
__device__ __forceinline__ Line make_line(int B, int pieces, long long min_piece, long long* sh, Weight weight) {
  constexpr int kW = kThreads / 32;
  long long v = 0;
  for (int b = threadIdx.x; b < B; b += kThreads) v += weight(b);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = v;
  __syncthreads();
  Line l;
  l.total = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) l.total += sh[w];
  l.piece = quotient(l.total + pieces - 1, pieces);
  if (l.piece < min_piece) l.piece = min_piece;
  return l;
}

// Sequence that holds point x of the line, and the point where it begins.  All threads get both.
template <int kThreads, typename Weight>
__device__ __forceinline__ void find_seq(int B, long long x, long long* sh, Weight weight, int& b_out,
                                         long long& first_out) {
  constexpr int kW = kThreads / 32;
  long long before = 0;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const long long mine = b < B ? weight(b) : 0;
    long long upto = mine;  // inclusive sum over the warp
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += y;
    }
    __syncthreads();
    if (threadIdx.x == 0) sh[kW] = -1;
    if (lane == 31) sh[warp] = upto;
    __syncthreads();
    long long base = before, all = 0;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      if (w < warp) base += sh[w];
      all += sh[w];
    }
    const long long end = base + upto;
    if (x < end && x >= end - mine) {
      sh[kW] = b;
      sh[kW + 1] = end - mine;
    }
    __syncthreads();
    if (sh[kW] >= 0) {
      b_out = (int)sh[kW];
      first_out = sh[kW + 1];
      return;
    }
    before += all;
  }
  b_out = -1;
  first_out = 0;
}

// Both at once for piece `index`: the line, and the sequence that holds the piece's first point (or -1).
template <int kThreads, typename Weight>
__device__ __forceinline__ Line find_piece(int B, int pieces, long long min_piece, int index, long long* sh,
                                           Weight weight, int& b_out, long long& first_out) {
  constexpr int kW = kThreads / 32;
  b_out = -1;
  first_out = 0;
  if (B > kThreads) {
    const Line l = make_line<kThreads>(B, pieces, min_piece, sh, weight);
    if (l.piece * index < l.total) find_seq<kThreads>(B, l.piece * index, sh, weight, b_out, first_out);
    return l;
  }
  // one look at the lengths: a thread per sequence
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const long long mine = (int)threadIdx.x < B ? weight((int)threadIdx.x) : 0;
  long long end = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, end, off);
    if (lane >= off) end += y;
  }
  if (lane == 31) sh[warp] = end;
  if (threadIdx.x == 0) sh[kW] = -1;
  __syncthreads();
  Line l;
  l.total = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    if (w < warp) end += sh[w];
    l.total += sh[w];
  }
  l.piece = quotient(l.total + pieces - 1, pieces);
  if (l.piece < min_piece) l.piece = min_piece;
  const long long x = l.piece * index;
  if (x < end && x >= end - mine) {
    sh[kW] = (int)threadIdx.x;
    sh[kW + 1] = end - mine;
  }
  __syncthreads();
  b_out = (int)sh[kW];
  first_out = sh[kW + 1];
  return l;
}

// ---------------------------------------------------------------- 4-bit codes as bf16
// Two codes (bits [0,4) and [16,20) of x) as bf16 code - 8: 0x4300 | c is 128 + c.
__device__ __forceinline__ uint32_t less_136(uint32_t y) {
  const __nv_bfloat162 off = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));
  const __nv_bfloat162 z = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&y), off);
  return *reinterpret_cast<const uint32_t*>(&z);
}
// 128 + code.  One instruction: written with two constants in C it becomes two, and these set the kernels' pace.
__device__ __forceinline__ uint32_t codes_128(uint32_t x) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "r"(0x000f000fu), "r"(0x43004300u));  // (x & a) | b
  return y;
}
__device__ __forceinline__ uint32_t codes_bf16(uint32_t x) { return less_136(codes_128(x)); }

}  // namespace s2
