// s2_cache_join.cuh -- adding up the partial sums of a unit of cached attention
// that several CTAs computed, one row behind the other (s2_cache_attn.cu;
// s2_cache_chunk.cu lays them transposed, and has its own loop).
//
// A piece leaves for each row O (D floats, not divided), then its maximum
// score, the sum of its weights and what O is to be divided by; in the order of
// the pieces
//     m = max m_p,  o = sum 2^(m_p - m) O_p / sum 2^(m_p - m) d_p,
// and lse from the sum of weights.
// A row has seen no key exactly where its sum of weights is 0.  Its maximum does not tell: a maximum leaves NaN out, so
// that of NaN scores alone is -inf too, while their sum is NaN and has to come through.
// What bounds it is the latency of reading them, so all of a warp's loads are
// asked for before the first is used: with up to 8 pieces a warp takes a row,
// with more a CTA does, its warps sharing the pieces.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sm100_ptx.cuh"

namespace s2 {

// What scores are taken from for a maximum m: 0 where that is infinite, so that no infinity is taken from another (a
// score of inf then has a weight of inf, and lse is inf as its definition says).
__device__ __forceinline__ float base_of(float m) { return fabsf(m) == INFINITY ? 0.f : m; }
// 1 / d of a row whose weights' sum is l.  l = 0: the token at `place` sees no key (place < 0) and gets 0, or its scores
// are all -inf, and o is 0 / 0.
__device__ __forceinline__ float row_scale(float l, float d, int place) {
  return l != 0.f ? 1.f / d : place < 0 ? 0.f : NAN;
}
// lse in natural logarithms; -inf of a row without keys.
__device__ __forceinline__ float row_lse(float m, float l) { return (m + log2f(l)) * 0.69314718055994531f; }

constexpr int kJoinThreads = 256;
constexpr int kJoinBatch = 8;  // pieces that a warp asks for at once

// Floats of a row's partial sums.
template <int D>
constexpr int kPartial = D + 4;

// A unit that the end of a piece cuts; rows = 0: it cuts none.
struct alignas(16) JoinCut {
  int rows;          // query rows of the unit
  int nth, helpers;  // which of the unit's cuts this is, and how many there are
  int begin;         // piece in which the unit begins: its sums are in the piece's second slot, the others' in the first
  int p0, p1;        // pieces that hold sums
  int tok, row0;     // row i is query row row0 + i of the heads from `head` on, from token tok on
  int head;
  int place;         // of token tok
  int pad[2];
};
constexpr size_t kCutBytes = 8192;  // of a workspace, before the sums, where pieces note what they cut

template <int D>
struct JoinShared {
  float m[kJoinThreads / 32], l[kJoinThreads / 32], d[kJoinThreads / 32];
  alignas(16) float o[kJoinThreads / 32][D];
};

// Sum of pieces p, p + by, .. <= p1 of one row: a lane holds channels [lane·D/32, ..).
template <int D, typename Part>
__device__ __forceinline__ void join_pieces(int p, int by, int p1, int row, Part part, float& m, float& l,
                                            float& d, float (&o)[D / 32]) {
  constexpr int kV = D / 32;
  const int lane = threadIdx.x % 32;
  m = -INFINITY;
  l = d = 0.f;
#pragma unroll
  for (int z = 0; z < kV; ++z) o[z] = 0.f;
  for (; p <= p1; p += kJoinBatch * by) {
    float4 ml[kJoinBatch];
    float v[kJoinBatch][kV];
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) {
      ml[i] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll
      for (int z = 0; z < kV; ++z) v[i][z] = 0.f;
      if (p + i * by <= p1) {
        const float* from = part(p + i * by, row);
        ml[i] = *reinterpret_cast<const float4*>(from + D);
        if constexpr (kV == 4) {
          const float4 t = *reinterpret_cast<const float4*>(from + 4 * lane);
          v[i][0] = t.x, v[i][1] = t.y, v[i][2] = t.z, v[i][3] = t.w;
        } else {
          const float2 t = *reinterpret_cast<const float2*>(from + 2 * lane);
          v[i][0] = t.x, v[i][1] = t.y;
        }
      }
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) top = fmaxf(top, ml[i].x);
    const float base = base_of(top), f = ex2(m - base);
    l *= f;
    d *= f;
#pragma unroll
    for (int z = 0; z < kV; ++z) o[z] *= f;
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) {
      const float g = ex2(ml[i].x - base);
      l = fmaf(ml[i].y, g, l);
      d = fmaf(ml[i].z, g, d);
#pragma unroll
      for (int z = 0; z < kV; ++z) o[z] = fmaf(v[i][z], g, o[z]);
    }
    m = top;
  }
}

// Rows of a cut unit, shared out over the CTAs of its cuts.
template <int D>
__device__ __forceinline__ void join_rows(JoinShared<D>& sh, const JoinCut u, const float* partial, int slot_rows,
                                          int g, int heads, __nv_bfloat16* o_all, float* lse) {
  constexpr int kW = kJoinThreads / 32, kV = D / 32;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (u.rows == 0) return;
  const int nth = u.nth, helpers = u.helpers;
  const bool narrow = u.p1 - u.p0 < kJoinBatch;
  const int first = narrow ? nth * kW + warp : nth, by = narrow ? helpers * kW : helpers;
  auto part = [&](int p, int row) {
    return partial + ((size_t)(2 * p + (p == u.begin)) * slot_rows + row) * kPartial<D>;
  };
  for (int i = first; i < u.rows; i += by) {
    float m, l, div, o[kV];
    join_pieces<D>(narrow ? u.p0 : u.p0 + warp, narrow ? 1 : kW, u.p1, i, part, m, l, div, o);
    if (!narrow) {
      __syncthreads();
      if (lane == 0) sh.m[warp] = m, sh.l[warp] = l, sh.d[warp] = div;
#pragma unroll
      for (int z = 0; z < kV; ++z) sh.o[warp][kV * lane + z] = o[z];
      __syncthreads();
      if (warp != 0) continue;
#pragma unroll
      for (int w = 1; w < kW; ++w) m = fmaxf(m, sh.m[w]);
      l = div = 0.f;
#pragma unroll
      for (int z = 0; z < kV; ++z) o[z] = 0.f;
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const float f = ex2(sh.m[w] - base_of(m));
        l = fmaf(sh.l[w], f, l);
        div = fmaf(sh.d[w], f, div);
#pragma unroll
        for (int z = 0; z < kV; ++z) o[z] = fmaf(sh.o[w][kV * lane + z], f, o[z]);
      }
    }
    const int at = u.row0 + i;
    const float inv = row_scale(l, div, u.place + at / g);
    const size_t out = (size_t)(u.tok + at / g) * heads + u.head + at % g;
    uint32_t* dst = reinterpret_cast<uint32_t*>(o_all + out * D) + lane * (kV / 2);
    if constexpr (kV == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
    else
      *dst = pack_bf16(o[0] * inv, o[1] * inv);
    if (lse && lane == 0) lse[out] = row_lse(m, l);
  }
}

}  // namespace s2
