// s2_cache_append.cu -- filling a paged cache of keys and values, and reading
// its rows back.
//
// Append: the new keys (and, beside them, the queries) are rotated to their
// positions as in s2_rope.cu and keys and values go to their rows of the
// cache, in bf16 or packed to 4 bits, in one pass over q, k and v, and no
// rotated copy of k is written.  HBM bounds the pass into bf16 rows, the
// rotation rides along (34,500 tokens of 32 + 8 heads of 128 channels, 848 MB:
// 140 us); into 4-bit rows packing's instructions do (issue slots 73% taken;
// 18,900 tokens 79 us, HBM's part 62), for a few tokens latency does.  Reading
// 4-bit rows back is bound by instructions too (the same 18,900 tokens 24 us, HBM's
// part 15; ALU 64%, issue 63%: a row's place by division, codes to numbers).
//
// Work: a CTA takes one token, or 4.  Their places, pages and angles come first
// (one warp per token finds its sequence, one thread per (token, pair) its
// angle), then D/16 lanes take a row of one head: lane i the channels
// [8i, 8i + 8) and [D/2 + 8i, D/2 + 8i + 8), which are 8 rotation pairs and, in
// 4 bits, 8 bytes.  A 4-bit row needs its extremes before its codes: they
// come from shuffles among those lanes, so the row is read once.
//
// The angle in turns, pos·scale·base^(-2j/D) / 2π, is formed and reduced to
// [-1/2, 1/2] in 64 bits, its sine and cosine taken there and rounded to 32.
// The rotation is done in 32 bits and rounded once to bf16.  4-bit codes are
// made from the bf16 row, so both formats hold the same rotated row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "s2_cache.cuh"
#include "s2_kernels.h"
#include "sm100_ptx.cuh"

namespace s2 {

namespace {

constexpr int kThreads = 256;
// Calls of up to this many tokens give each a CTA: all of them are resident at once, and a token's rows go by in the
// fewest turns (32 + 8 heads, 64 tokens: append 4.3 us with 1 token to a CTA, 6.7 with 4; 600 tokens 6.1 and 7.0).
// Beyond, what a CTA does before its rows is shared by 4 tokens (2400 tokens in 4 bits: 15.1 us, 18.9 with 1).
constexpr int kLoneTokens = 5 * 148;

// Sequence of packed token t: the number of sequences whose new tokens end at or before t.
// Whole warp; B when no sequence holds it.
__device__ __forceinline__ int seq_of_token(const CacheArgs& c, int t, int lane) {
  if (!c.starts) return t;
  int n = 0;
  for (int b = lane; b < c.B; b += 32) n += c.starts[b + 1] <= t;
  return __reduce_add_sync(0xffffffffu, n);
}

// Places and pages of the CTA's tokens; place < 0 or ok false: nothing is stored.
struct Token {
  int place;
  int page;
  bool mine;   // belongs to a sequence
  bool store;  // and has a row in the cache
};

template <int N>
__device__ __forceinline__ void find_tokens(const CacheArgs& c, int t0, Token* tok) {
  const int lane = threadIdx.x % 32;
  for (int x = threadIdx.x / 32; x < N; x += kThreads / 32) {
    const int t = t0 + x;
    Token r{0, 0, false, false};
    if (t < c.T) {
      const int b = seq_of_token(c, t, lane);
      if (b < c.B) {
        const Seq s = load_seq(c, b);
        if (t >= s.first && t - s.first < s.n) {
          r.place = s.len - s.n + (t - s.first);
          r.mine = true;
          if (r.place >= 0) {
            const int page = c.table[(size_t)b * c.width + (r.place >> c.log2s)];
            r.store = (unsigned)page < (unsigned long long)c.pages;
            r.page = r.store ? page : 0;
            if (!r.store && lane == 0) atomicOr(c.status, kCacheFlag);
          }
        }
      }
    }
    if (lane == 0) tok[x] = r;
  }
}

struct Row {
  float lo[8], hi[8];  // channels [8i, 8i + 8) and [D/2 + 8i, ..)
};

__device__ __forceinline__ void unpack8(const uint4& raw, float* x) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes min(rint(a / s), 15) of a thread's 16 numbers a = x - min, as its 8 bytes.  Numbers of bf16 often lie right
// between two codes, so the quotient must be the correctly rounded one: from the correctly rounded reciprocal y,
// q = a y and q + (a - q s) y, the remainder exact (Markstein's theorem), a third of a division's instructions.
// Added to 1.5·2^23 its low bits are the rounded quotient, with no conversion (those run at a quarter of the rate),
// and eight sums' bits added up in their places, less eight times the constant's, are a word.
__device__ __forceinline__ uint2 codes_of(const Row& a, float s) {
  constexpr float kMagic = 12582912.f;        // 0x4b400000
  constexpr uint32_t kBits = 0x4b400000u * 0x11111111u;
  const float y = __frcp_rn(s);
  auto place = [&](float x) -> uint32_t {
    const float q = x * y;
    return __float_as_uint(fmaf(fmaf(-q, s, x), y, q) + kMagic);
  };
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t sum = 0u - kBits;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sum += place(a.lo[4 * h + i]) * (1u << (8 * i)) + place(a.hi[4 * h + i]) * (16u << (8 * i));
    w[h] = sum;
  }
  if (s < 1e-30f) {  // remainders or the reciprocal would leave the range of 32 bits
    w[0] = w[1] = 0u;
    for (int i = 0; i < 8; ++i) {
      const uint32_t lo = (uint32_t)fminf(rintf(__fdiv_rn(a.lo[i], s)), 15.f);
      const uint32_t hi = (uint32_t)fminf(rintf(__fdiv_rn(a.hi[i], s)), 15.f);
      w[i / 4] |= (lo | (hi << 4)) << (8 * (i % 4));
    }
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ __nv_bfloat162 as_pair(uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }

// Packs a row held by LANES lanes (bf16 values) to 4 bits: this lane's 8 bytes and the row's (scale, min).
// A row with a NaN or an infinity, or whose scale is none, reads back as NaN.
template <int LANES>
__device__ __forceinline__ void pack_row(const uint4& lo, const uint4& hi, uint2& codes, uint32_t& pair) {
  // extremes of pairs of numbers; 0 times a number that is none is none
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  const __nv_bfloat162 zero = as_pair(0u);
  __nv_bfloat162 mn2 = as_pair(w[0]), mx2 = mn2, broken = zero;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mn2 = __hmin2(mn2, as_pair(w[i]));
    mx2 = __hmax2(mx2, as_pair(w[i]));
    broken = __hfma2(as_pair(w[i]), zero, broken);
  }
  float mn = fminf(__low2float(mn2), __high2float(mn2)), mx = fmaxf(__low2float(mx2), __high2float(mx2));
  int good = __low2float(broken) == 0.f && __high2float(broken) == 0.f;
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    good &= __shfl_xor_sync(0xffffffffu, good, off);
  }
  // the scale is rounded to bf16 (8 bits) before the codes are chosen, so the rounding moves the grid
  // (by 2^-8 of it at most, 0.06 of a step at its end) and not the error of a value
  __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(mx - mn, 15.0f));
  __nv_bfloat16 mb = __float2bfloat16_rn(mn);  // exact: the row is bf16
  const float s = __bfloat162float(sb);
  good &= s < INFINITY;
  codes = make_uint2(0u, 0u);
  if (good && s > 0.f) {
    Row x;
    unpack8(lo, x.lo);
    unpack8(hi, x.hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) x.lo[i] -= mn, x.hi[i] -= mn;
    codes = codes_of(x, s);
  }
  if (!good) sb = mb = __float2bfloat16_rn(NAN);
  pair = (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(mb) << 16);
}

}  // namespace

// A thread's way through the rows of the CTA's tokens: row `r` of token `x`, kRows further each time.
struct RowAt {
  int x, r;
  __device__ __forceinline__ void next(int by, int per_token) {
    r += by;
    while (r >= per_token) {
      r -= per_token;
      ++x;
    }
  }
};

// Rows of a token in order: H query heads (none without q), Hkv key heads, Hkv value heads.  Where a row
// comes from does not depend on its sequence: the first rows are on their way before the tokens are found,
// and each next row while the last one is worked on.
// Six CTAs an SM hold 40 registers a thread, enough for bf16 rows (34,500 tokens of 32 and 8 heads 139.7 us, with five
// 141.7, the HBM's 129); packing needs 48, so five (18,900 tokens 79.2 us; 82.6 as compiled without a bound, 82.2 with
// six, which spill).
template <int D, bool Q4, bool kRotate, int kTok>
__global__ void __launch_bounds__(kThreads, Q4 ? 5 : 6)
    s2_cache_append_kernel(const __grid_constant__ CacheArgs c, const __grid_constant__ AppendIn in) {
  constexpr int kHalf = D / 2, kLanes = D / 16, kRows = kThreads / kLanes;
  __shared__ Token tok[kTok];
  __shared__ __align__(16) float2 cs[kTok][kHalf];
  const int t0 = blockIdx.x * kTok;
  const int here = min(kTok, c.T - t0);
  const int per_token = in.q_heads + 2 * c.heads;
  const int lane = threadIdx.x % kLanes;
  RowAt at{0, 0};
  at.next(threadIdx.x / kLanes, per_token);
  uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
  auto load = [&](const RowAt& a) {
    if (a.x >= here) return;
    const int v0 = in.q_heads + c.heads;
    const __nv_bfloat16* src = (a.r < in.q_heads ? in.q + (size_t)(t0 + a.x) * in.ldq + (size_t)a.r * D
                                : a.r < v0       ? in.k + (size_t)(t0 + a.x) * in.ldk + (size_t)(a.r - in.q_heads) * D
                                                 : in.v + (size_t)(t0 + a.x) * in.ldv + (size_t)(a.r - v0) * D) +
                               8 * lane;
    lo = *reinterpret_cast<const uint4*>(src);
    hi = *reinterpret_cast<const uint4*>(src + kHalf);
  };
  load(at);
  find_tokens<kTok>(c, t0, tok);
  __syncthreads();
  if constexpr (kRotate) {
    for (int i = threadIdx.x; i < kTok * kHalf; i += kThreads) {
      const int x = i / kHalf, j = i % kHalf;
      if (tok[x].mine) {
        const int pos = in.positions ? in.positions[t0 + x] : tok[x].place;
        const double turns = (double)pos * in.turns[j];
        double s, co;
        sincospi(2.0 * (turns - rint(turns)), &s, &co);
        cs[x][j] = make_float2((float)co, (float)s);
      }
    }
    __syncthreads();
  }
  // whole warps go around together (the packing's shuffles need all lanes)
  for (int w0 = 0; w0 < here * per_token; w0 += kRows) {
    const RowAt now = at;
    Row row;
    unpack8(lo, row.lo);
    unpack8(hi, row.hi);
    at.next(kRows, per_token);
    load(at);
    const bool is_q = now.r < in.q_heads, is_v = now.r >= in.q_heads + c.heads;
    const int h = is_q ? now.r : is_v ? now.r - in.q_heads - c.heads : now.r - in.q_heads;
    const bool live = now.x < here && (is_q ? tok[now.x].mine : tok[now.x].store);
    if (kRotate && live && !is_v) {
      const float4* angles = reinterpret_cast<const float4*>(&cs[now.x][8 * lane]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 a4 = angles[i / 2];
        const float co = i % 2 ? a4.z : a4.x, si = i % 2 ? a4.w : a4.y;
        // products rounded one by one, as plain 32-bit arithmetic does it: a value at a rounding border
        // must not depend on the compiler's choice, since 4-bit codes are made from it
        const float a = __fsub_rn(__fmul_rn(row.lo[i], co), __fmul_rn(row.hi[i], si));
        const float b = __fadd_rn(__fmul_rn(row.hi[i], co), __fmul_rn(row.lo[i], si));
        row.lo[i] = a;
        row.hi[i] = b;
      }
    }
    const uint4 out_lo = pack8(row.lo), out_hi = pack8(row.hi);
    if (live && (!Q4 || is_q)) {
      __nv_bfloat16* dst = is_q ? in.q_out + ((size_t)(t0 + now.x) * in.q_heads + h) * D
                                : static_cast<__nv_bfloat16*>(is_v ? c.v : c.k) +
                                      row_of(c, tok[now.x].page, h, tok[now.x].place) * D;
      *reinterpret_cast<uint4*>(dst + 8 * lane) = out_lo;
      *reinterpret_cast<uint4*>(dst + kHalf + 8 * lane) = out_hi;
    }
    if constexpr (Q4) {
      if (!__any_sync(0xffffffffu, live && !is_q)) continue;
      uint2 codes;
      uint32_t pair;
      pack_row<kLanes>(out_lo, out_hi, codes, pair);
      if (live && !is_q) {
        const size_t to = row_of(c, tok[now.x].page, h, tok[now.x].place);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? c.v : c.k) + to * kHalf + 8 * lane) = codes;
        if (lane == 0) static_cast<uint32_t*>(is_v ? c.v_scale : c.k_scale)[to] = pair;
      }
    }
  }
}

// The inverse: rows of the batch's tokens, k and v [T, Hkv, D] in bf16 (one rounding from 4 bits).
// Tokens of no sequence, or with no row in the cache, are left as they are.
template <int D, bool Q4, int kTokens>
__global__ void __launch_bounds__(kThreads) s2_cache_read_kernel(const __grid_constant__ CacheArgs c,
                                                                 __nv_bfloat16* __restrict__ k_out,
                                                                 __nv_bfloat16* __restrict__ v_out) {
  constexpr int kHalf = D / 2, kLanes = D / 16, kRows = kThreads / kLanes;
  __shared__ Token tok[kTokens];
  const int t0 = blockIdx.x * kTokens;
  find_tokens<kTokens>(c, t0, tok);
  __syncthreads();
  const int per_token = 2 * c.heads;
  const int lane = threadIdx.x % kLanes;
#pragma unroll 8
  for (int w = threadIdx.x / kLanes; w < kTokens * per_token; w += kRows) {
    const int x = w / per_token, r = w % per_token;
    if (!tok[x].store) continue;
    const bool is_v = r >= c.heads;
    const int h = is_v ? r - c.heads : r;
    const size_t at = row_of(c, tok[x].page, h, tok[x].place);
    __nv_bfloat16* dst = (is_v ? v_out : k_out) + ((size_t)(t0 + x) * c.heads + h) * D;
    uint4 lo, hi;
    if constexpr (Q4) {
      const uint2 codes =
          *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(is_v ? c.v : c.k) + at * kHalf + 8 * lane);
      const float2 p = q4_pair(static_cast<const uint32_t*>(is_v ? c.v_scale : c.k_scale)[at]);
      Row row;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = ((i < 4 ? codes.x : codes.y) >> (8 * (i % 4))) & 0xffu;
        // scale·code is exact (8 + 4 bits), so this is one rounding to 32 bits
        row.lo[i] = fmaf(p.x, (float)(b & 15u), p.y);
        row.hi[i] = fmaf(p.x, (float)(b >> 4), p.y);
      }
      lo = pack8(row.lo);
      hi = pack8(row.hi);
    } else {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? c.v : c.k) + at * D + 8 * lane;
      lo = *reinterpret_cast<const uint4*>(src);
      hi = *reinterpret_cast<const uint4*>(src + kHalf);
    }
    *reinterpret_cast<uint4*>(dst + 8 * lane) = lo;
    *reinterpret_cast<uint4*>(dst + kHalf + 8 * lane) = hi;
  }
}

template <int D, bool Q4, int kTok>
static int append_impl(const CacheArgs& c, const AppendIn& in, bool rotate, cudaStream_t stream) {
  const unsigned grid = (unsigned)((c.T + kTok - 1) / kTok);
  if (rotate)
    s2_cache_append_kernel<D, Q4, true, kTok><<<grid, kThreads, 0, stream>>>(c, in);
  else
    s2_cache_append_kernel<D, Q4, false, kTok><<<grid, kThreads, 0, stream>>>(c, in);
  return (int)cudaGetLastError();
}

template <int D, bool Q4>
static int append_tokens(const CacheArgs& c, const AppendIn& in, bool rotate, cudaStream_t stream) {
  return c.T <= kLoneTokens ? append_impl<D, Q4, 1>(c, in, rotate, stream) : append_impl<D, Q4, 4>(c, in, rotate, stream);
}

int launch_cache_append(const CacheArgs& c, const AppendIn& in, int D, bool q4, bool rotate, cudaStream_t stream) {
  if (D == 64) return q4 ? append_tokens<64, true>(c, in, rotate, stream) : append_tokens<64, false>(c, in, rotate, stream);
  return q4 ? append_tokens<128, true>(c, in, rotate, stream) : append_tokens<128, false>(c, in, rotate, stream);
}

template <int D, bool Q4>
static int read_impl(const CacheArgs& c, void* k_out, void* v_out, cudaStream_t stream) {
  auto* k = static_cast<__nv_bfloat16*>(k_out);
  auto* v = static_cast<__nv_bfloat16*>(v_out);
  // As for append (32 heads, 64 tokens in 4 bits: 3.6 us with 1 token to a CTA, 6.1 with 4; 8 heads, 2400 tokens 6.9
  // and 5.4), and CTAs of few heads take 8 tokens, if that leaves CTAs for all SMs (8 heads, 8192 tokens in 4 bits:
  // 10.5 us with 8, 11.4 with 4; 32 heads, 8192 tokens: 34.7 with 8 or 4 in 4 bits, 50.6 and 46.9 in bf16).
  if (c.T <= kLoneTokens)
    s2_cache_read_kernel<D, Q4, 1><<<(unsigned)c.T, kThreads, 0, stream>>>(c, k, v);
  else if (c.heads < 16 && (int64_t)c.T * c.heads >= 1 << 16)
    s2_cache_read_kernel<D, Q4, 8><<<(unsigned)((c.T + 7) / 8), kThreads, 0, stream>>>(c, k, v);
  else
    s2_cache_read_kernel<D, Q4, 4><<<(unsigned)((c.T + 3) / 4), kThreads, 0, stream>>>(c, k, v);
  return (int)cudaGetLastError();
}

int launch_cache_read(const CacheArgs& c, int D, bool q4, void* k_out, void* v_out, cudaStream_t stream) {
  if (D == 64) return q4 ? read_impl<64, true>(c, k_out, v_out, stream) : read_impl<64, false>(c, k_out, v_out, stream);
  return q4 ? read_impl<128, true>(c, k_out, v_out, stream) : read_impl<128, false>(c, k_out, v_out, stream);
}

}  // namespace s2
