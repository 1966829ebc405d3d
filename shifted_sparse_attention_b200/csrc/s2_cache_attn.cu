// s2_cache_attn.cu -- attention of a few new tokens over a paged cache.
//
// For new token t of sequence b at place p, head h of key/value head h / g:
//     o = sum_{j <= p} softmax_j(q·k_j / sqrt(D)) v_j,   lse = ln sum exp.
// From a 4-bit cache, with k_j = mk + sk·ck:
//     q·k_j       = sk (q·(128 + ck_j)) + (mk - 128 sk) sum(q)  (and 2^-5 of it: s2_cache.cuh),
//     sum p_j v_j = sum (p_j sv_j)(cv_j - 8) + sum p_j (mv_j + 8 sv_j),
// so the matrix products see whole numbers, which bf16 holds as they are, and
// nothing of a row is rounded (values centred: rounded weights then meet small
// numbers).
//
// Bound: HBM (each row of the cache is read once, and serves the g·n rows of
// queries that share it).  Everything else is arranged around keeping loads
// in flight:
// - a unit is (sequence, key/value head, block of 8·NR query rows); its keys
//   are cut into steps of kStep keys.  All units' steps form one line, cut
//   into equal pieces, one per CTA, so sequences of any lengths load all SMs
//   alike; a unit cut by a border leaves partial sums (max, sum, O) that
//   a second launch adds up in a fixed order.
//   Short units (cut_units below) are not cut: a CTA takes one, or a cluster's
//   CTAs take equal parts of one and add their sums up through each other's
//   shared memory, in one launch.
// - a warp takes every fourth step of its CTA's piece by itself: loads go from
//   global memory straight to the registers that mma.sync reads as its A
//   operand (S^T = K Q^T and O^T = V^T P^T, so keys fill the 16-row side and
//   the few query rows the 8-column side), with no shared memory and no
//   barrier in the loop.  K of the next step is asked for when this step's
//   scores are done, V when its products are.
// - channels and keys may come in any order inside a product as long as both
//   operands agree, so every lane loads 16 contiguous bytes (8 in 4 bits) of a
//   row; V's pairs along the keys are put together with byte permutes, the
//   weights' with one 8x8 transposition (movmatrix).
// - the running maximum moves only when a score passes it by more than 8 (a
//   factor 256), which one vote per step tells; sums are in 32 bits.  The
//   weights are rounded to bf16 for the product (2^-8 of each at most); O is
//   divided by the sum of the rounded ones where that is to be had (bf16 rows),
//   so that it stays a mean of values, and lse comes from the unrounded sum.
// Measured (D 128): 64 sequences of 17 to 8192 keys, 32 heads on 8 key heads,
// 1.09 GB, 172 us, 0.96 of the measured copy rate; one of 32768 keys 25.2 us
// (HBM's part 20.5); 4 bits, 48 sequences of 33 to 4096 keys, 32 key heads, 433 MB,
// 111 us (HBM's part 66).  There no pipe is near its limit (ALU 56%, issue 56%, HBM
// 47%): of the time that a warp is not issuing, 28% goes to the fixed latencies of
// its own last instruction, 26% to loads, 15% to other warps' turns, 14% to a busy
// ALU, with 16 warps of 128 registers on an SM.
#include <climits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "s2_cache.cuh"
#include "s2_cache_join.cuh"
#include "s2_kernels.h"
#include "sm100_ptx.cuh"

namespace s2 {

namespace {

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The caches are read once: past L1, and first to leave L2.
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_stream4(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// Shared memory of the cluster's CTA `rank` at this CTA's address.
__device__ __forceinline__ float4 ld_cluster16(const void* p, int rank) {
  float4 v;
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
// All threads of all of the cluster's CTAs; what they wrote before is seen by all after.  Not the .aligned form: that one
// wants a warp's lanes together, and they come from loops that end at different turns (a row of 64 channels is half a
// warp's) and from stores that one lane in 16 or 32 makes.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}

// Registers of one 16-key block of K and of V in the order the products take them.
template <int D, bool Q4>
struct KeyRegs;
template <int D>
struct KeyRegs<D, false> {
  uint4 w[D / 32][2];  // [32-channel block][key r / r + 8]: channels 32i + 8c ..
};
template <int D>
struct KeyRegs<D, true> {
  uint32_t w[2][D / 32];  // [key r / r + 8]: D/8 bytes from byte (D/8)c
  uint32_t pair[2];
};
template <int D, bool Q4>
struct ValueRegs;
template <int D>
struct ValueRegs<D, false> {
  uint4 w[4][D / 64];  // [key 2c, 2c+1, 2c+8, 2c+9][64-channel block]: channels 64i + 8r ..
};
template <int D>
struct ValueRegs<D, true> {
  uint32_t w[4][D / 64];  // D/16 bytes from byte (D/16)r
  uint32_t pair[2];       // of keys r, r + 8
};

// A lane's place in a block of rows: bytes from the block's first row, for keys and for values.
template <int D, bool Q4>
__device__ __forceinline__ void load_keys(KeyRegs<D, Q4>& x, const uint8_t* rows, const uint8_t* pairs) {
  constexpr int kRow = Q4 ? D / 2 : 2 * D;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* p = rows + 8 * u * kRow;
    if constexpr (Q4) {
      if constexpr (D == 128) {
        const uint4 v = ld_stream16(p);
        x.w[u][0] = v.x, x.w[u][1] = v.y, x.w[u][2] = v.z, x.w[u][3] = v.w;
      } else {
        const uint2 v = ld_stream8(p);
        x.w[u][0] = v.x, x.w[u][1] = v.y;
      }
      x.pair[u] = ld_stream4(pairs + 32 * u);
    } else {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) x.w[i][u] = ld_stream16(p + 64 * i);
    }
  }
}

template <int D, bool Q4>
__device__ __forceinline__ void load_values(ValueRegs<D, Q4>& x, const uint8_t* rows, const uint8_t* pairs) {
  constexpr int kRow = Q4 ? D / 2 : 2 * D;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint8_t* p = rows + ((u & 1) + 8 * (u >> 1)) * kRow;
    if constexpr (Q4) {
      if constexpr (D == 128) {
        const uint2 v = ld_stream8(p);
        x.w[u][0] = v.x, x.w[u][1] = v.y;
      } else {
        x.w[u][0] = ld_stream4(p);
      }
    } else {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) x.w[u][i] = ld_stream16(p + 128 * i);
    }
  }
  if constexpr (Q4) {
#pragma unroll
    for (int u = 0; u < 2; ++u) x.pair[u] = ld_stream4(pairs + 32 * u);
  }
}

// Channel of row `r` (+ 8 when hi) of O^T's tile j: the order in which V's lanes load.
template <int D, bool Q4>
__device__ __forceinline__ int channel_of(int j, bool hi, int r) {
  if constexpr (Q4) return (D / 16) * r + j + (hi ? D / 2 : 0);
  if constexpr (D == 128) return 8 * r + j + (hi ? 64 : 0);
  return 8 * r + j + (hi ? 4 : 0);
}

// Steps of a unit of a sequence of len tokens; one for an empty sequence, whose rows are then written empty.
__host__ __device__ constexpr int steps_of(int len, int step) { return len > 0 ? (len + step - 1) / step : 1; }

// One block of query rows: units of sequence b are (kv head, block of 8·NR rows).
template <int NR>
__device__ __forceinline__ int row_blocks(int n, int g) {
  return (int)(((long long)n * g + 8 * NR - 1) / (8 * NR));
}

// Warps of a CTA.
constexpr int kW = 4;

// A unit takes kUnitSteps + steps of the line: what starting and ending it costs, then its steps.
// (Without the first, a piece of many short sequences took several times as long as the others.)
constexpr int kUnitSteps = 2 * kW;

template <int NR>
__device__ __forceinline__ long long seq_steps(const CacheArgs& c, const AttnIn& in, int b, int step, bool cut) {
  const Seq s = load_seq(c, b);
  return (long long)c.heads * row_blocks<NR>(s.n, in.g) * (cut ? steps_of(s.len, step) + kUnitSteps : 1);
}

}  // namespace

// 16-key blocks of a step: what a warp has in flight, against its registers.
template <bool Q4>
__host__ __device__ constexpr int step_blocks() { return Q4 ? 2 : 1; }

// CTAs on an SM: 12 warps of 168 registers for bf16 rows (16 of 128 spill: one sequence of 32768 keys took
// 28.7 us and not 23.1), 16 of 128 for 4-bit ones, 8 of 255 with two blocks of query rows.
template <bool Q4, int NR>
__host__ __device__ constexpr int ctas_per_sm() { return (NR == 2 ? 8 : Q4 ? 16 : 12) / kW; }

constexpr int kMaxCluster = 8;

template <int D, int NR>
struct DecodeShared {
  long long line[kW + 2];
  long long x0, x1;  // the CTA's piece [x0, x1) of the line: here and not in registers, which the keys need
  float m[kW][8 * NR], l[kW][8 * NR], div[kW][8 * NR];  // maximum, sum of weights, what O is divided by
  alignas(16) float4 all[8 * NR];                    // the same of the CTA, for its cluster (O is then in o[0])
  alignas(16) float o[kW][8 * NR][D + 4];
};

template <int D, bool Q4, int NR>
__global__ void __launch_bounds__(kW * 32, ctas_per_sm<Q4, NR>())
    s2_cache_decode_kernel(const __grid_constant__ CacheArgs c, const __grid_constant__ AttnIn in) {
  constexpr int kThreads = kW * 32;
  constexpr int kBlocks = step_blocks<Q4>();
  constexpr int kStep = 16 * kBlocks;
  constexpr int kRows = 8 * NR;
  constexpr int kTiles = D / 16;  // 16-channel tiles of O^T
  constexpr int kRowBytes = Q4 ? D / 2 : 2 * D;
  extern __shared__ __align__(16) uint8_t smem[];
  auto& sh = *reinterpret_cast<DecodeShared<D, NR>*>(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, r = lane / 4, cc = lane % 4;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may start its own set-up
  // cut units: each takes its steps of the line; whole units: one point each, and a CTA, or the CTAs of a cluster
  // together, take one unit
  const bool cut = in.pieces > 0;
  auto weight = [&](int i) { return seq_steps<NR>(c, in, i, kStep, cut); };
  int b;
  long long seq_first;
  const int index = (int)(blockIdx.x / (unsigned)in.cluster), rank = (int)(blockIdx.x % (unsigned)in.cluster);
  const Line line =
      find_piece<kThreads>(c.B, cut ? in.pieces : INT_MAX, in.min_piece, index, sh.line, weight, b, seq_first);
  if (line.piece * index >= line.total) return;  // (all of a cluster's CTAs do)
  if (threadIdx.x == 0) {
    sh.x0 = line.piece * index;
    sh.x1 = min(line.piece * (index + 1), line.total);
  }
  __syncthreads();
  // a lane's place in a block of 16 rows
  const uint8_t* const k_base = static_cast<const uint8_t*>(c.k) + r * kRowBytes + (Q4 ? (D / 8) : 16) * cc;
  const uint8_t* const v_base = static_cast<const uint8_t*>(c.v) + 2 * cc * kRowBytes + (Q4 ? (D / 16) : 16) * r;
  const uint8_t* const ks_base = static_cast<const uint8_t*>(c.k_scale) + 4 * r;
  const uint8_t* const vs_base = static_cast<const uint8_t*>(c.v_scale) + 4 * r;

  long long x = sh.x0;
  while (x < sh.x1) {
    Seq seq = load_seq(c, b);
    const int blocks = row_blocks<NR>(seq.n, in.g);
    const int steps = steps_of(seq.len, kStep);
    const int head = cut ? kUnitSteps : 0, span = cut ? steps + head : 1;
    if (x >= seq_first + (long long)c.heads * blocks * span) {  // this sequence is done
      seq_first += (long long)c.heads * blocks * span;
      ++b;
      continue;
    }
    const long long unit = quotient(x - seq_first, span);
    const long long unit_first = seq_first + unit * span + head;  // of its steps
    const int h = (int)quotient(unit, blocks), rb = (int)(unit - (long long)h * blocks);
    const int k0 = cut ? (int)max(0LL, x - unit_first) : (int)((unsigned)(steps * rank) / (unsigned)in.cluster);
    const int k1 = cut ? (int)min((long long)steps, sh.x1 - unit_first)
                       : (int)((unsigned)(steps * (rank + 1)) / (unsigned)in.cluster);
    x = unit_first + (cut ? steps : 1);
    if (cut && k1 <= k0) continue;
    const int slot = !cut || (k0 == 0 && k1 == steps) ? -1 : 2 * (int)blockIdx.x + (unit_first < sh.x0 ? 0 : 1);  // -1: whole

    // ---------------------------------------------------------- query rows
    // B operand of S^T: lane (r, cc) holds row r's channels as load_keys orders them
    uint32_t qf[NR][D / 16][2];
    float qsum[NR][2];
    int lim[NR][2];     // keys that the lane's two columns see
    int lim_all = seq.len;  // keys that every row sees
#pragma unroll
    for (int y = 0; y < NR; ++y) {
      const int row = rb * kRows + y * 8 + r;
      const bool live = row < seq.n * in.g;
      const __nv_bfloat16* p = in.q + (size_t)(seq.first + (live ? row / in.g : 0)) * in.ldq +
                               (size_t)(h * in.g + (live ? row % in.g : 0)) * D;
      float sum = 0.f;
      if constexpr (Q4) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            uint2 v = make_uint2(0u, 0u);
            if (live) v = *reinterpret_cast<const uint2*>(p + half * (D / 2) + (D / 8) * cc + 4 * w);
            // bytes 0, 2 and 1, 3 of a word of codes are taken together
            qf[y][2 * w + half][0] = __byte_perm(v.x, v.y, 0x5410);
            qf[y][2 * w + half][1] = __byte_perm(v.x, v.y, 0x7632);
            sum += __uint_as_float(v.x << 16) + __uint_as_float(v.x & 0xffff0000u) + __uint_as_float(v.y << 16) +
                   __uint_as_float(v.y & 0xffff0000u);
          }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
        for (int e = 0; e < 2; ++e) qsum[y][e] = kQ4Bias * __shfl_sync(0xffffffffu, sum, (2 * cc + e) * 4);
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (live) v = *reinterpret_cast<const uint4*>(p + 32 * i + 8 * cc);
          qf[y][2 * i][0] = v.x, qf[y][2 * i][1] = v.y, qf[y][2 * i + 1][0] = v.z, qf[y][2 * i + 1][1] = v.w;
        }
        qsum[y][0] = qsum[y][1] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = rb * kRows + y * 8 + 2 * cc + e;
        // rows of no token see every key; what they compute is not stored
        lim[y][e] = col < seq.n * in.g ? max(0, seq.len - seq.n + col / in.g + 1) : seq.len;
        lim_all = min(lim_all, lim[y][e]);
      }
    }
    lim_all = min(lim_all, __shfl_xor_sync(0xffffffffu, lim_all, 1));
    lim_all = min(lim_all, __shfl_xor_sync(0xffffffffu, lim_all, 2));

    // ---------------------------------------------------------- keys
    float acc[NR][kTiles][4];
    // maximum; sum of the weights; bf16 rows: of the weights as the product takes them, 4-bit rows: of weight·middle
    float m[NR][2], l[NR][2], vsum[NR][2];
#pragma unroll
    for (int y = 0; y < NR; ++y) {
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[y][j][i] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) m[y][e] = -INFINITY, l[y][e] = 0.f, vsum[y][e] = 0.f;
    }

    KeyRegs<D, Q4> kr[kBlocks];
    ValueRegs<D, Q4> vr[kBlocks];
    uint32_t rows[kBlocks];  // first rows of the next step's blocks (a cache's rows are counted in 32 bits)
    int k = k0 + warp;
    const int* const pages = c.table + (size_t)b * c.width;
    const int last_block = (seq.len - 1) & ~15, slot_mask = (1 << c.log2s) - 1;
    auto find_row = [&](int p) -> uint32_t {
      int page = pages[p >> c.log2s];
      if ((uint32_t)page >= (uint32_t)c.pages) {
        atomicOr(c.status, kCacheFlag);
        page = 0;
      }
      return ((((uint32_t)page * (uint32_t)c.heads + (uint32_t)h) << c.log2s)) + (uint32_t)(p & slot_mask);
    };
    // a block behind the last key is read from the last block instead: it lies in a page of the sequence
    auto find_rows = [&](int step) {
      rows[0] = find_row(step * kStep);
#pragma unroll
      for (int u = 1; u < kBlocks; ++u) {
        const int p = step * kStep + 16 * u;
        if (p > last_block)
          rows[u] = rows[u - 1];
        else
          rows[u] = c.log2s >= 5 && u % 2 ? rows[u - 1] + 16 : find_row(p);  // (steps of two blocks begin at even ones)
      }
    };
    if (seq.len > 0 && k < k1) {
      find_rows(k);
#pragma unroll
      for (int u = 0; u < kBlocks; ++u) load_keys(kr[u], k_base + (size_t)rows[u] * kRowBytes, ks_base + (size_t)rows[u] * 4);
#pragma unroll
      for (int u = 0; u < kBlocks; ++u) load_values(vr[u], v_base + (size_t)rows[u] * kRowBytes, vs_base + (size_t)rows[u] * 4);
      for (; k < k1; k += kW) {
        const int key0 = k * kStep;
        const bool more = k + kW < k1;
        if (more) find_rows(k + kW);
        // scores: keys r, r + 8 of each block by rows 2cc, 2cc + 1
        float s[NR][kBlocks][4];
#pragma unroll
        for (int u = 0; u < kBlocks; ++u) {
#pragma unroll
          for (int y = 0; y < NR; ++y) s[y][u][0] = s[y][u][1] = s[y][u][2] = s[y][u][3] = 0.f;
          if constexpr (Q4) {
#pragma unroll
            for (int w = 0; w < D / 32; ++w)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t a0 = codes_128(kr[u].w[0][w] >> (4 * half));
                const uint32_t a1 = codes_128(kr[u].w[1][w] >> (4 * half));
                const uint32_t a2 = codes_128(kr[u].w[0][w] >> (4 * half + 8));
                const uint32_t a3 = codes_128(kr[u].w[1][w] >> (4 * half + 8));
                // a word's bytes 0, 2 are channels 4w, 4w + 2: qf's first pair
#pragma unroll
                for (int y = 0; y < NR; ++y) {
                  const uint32_t q01 = qf[y][2 * w + half][0], q23 = qf[y][2 * w + half][1];
                  mma16816(s[y][u], a0, a1, a2, a3, q01, q23);
                }
              }
          } else {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              const uint4 a = kr[u].w[i][0], d = kr[u].w[i][1];
#pragma unroll
              for (int y = 0; y < NR; ++y) {
                mma16816(s[y][u], a.x, d.x, a.y, d.y, qf[y][2 * i][0], qf[y][2 * i][1]);
                mma16816(s[y][u], a.z, d.z, a.w, d.w, qf[y][2 * i + 1][0], qf[y][2 * i + 1][1]);
              }
            }
          }
          if constexpr (Q4) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const float2 pr = q4_key(q4_pair(kr[u].pair[t]));
#pragma unroll
              for (int y = 0; y < NR; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e) s[y][u][2 * t + e] = fmaf(s[y][u][2 * t + e], pr.x, pr.y * qsum[y][e]);
            }
          }
        }
        if (more) {
#pragma unroll
          for (int u = 0; u < kBlocks; ++u) load_keys(kr[u], k_base + (size_t)rows[u] * kRowBytes, ks_base + (size_t)rows[u] * 4);
        }
        // masks, only where some row or the sequence ends in the step
        if (key0 + kStep > lim_all) {
#pragma unroll
          for (int u = 0; u < kBlocks; ++u) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int key = key0 + 16 * u + r + 8 * t;
#pragma unroll
              for (int y = 0; y < NR; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (key >= lim[y][e]) s[y][u][2 * t + e] = -INFINITY;
              if constexpr (Q4) {
                if (key >= seq.len) vr[u].pair[t] = 0u;
              }
            }
            // rows behind the sequence hold anything; their weight is 0 and must stay so
            if constexpr (!Q4) {
#pragma unroll
              for (int t = 0; t < 4; ++t)
                if (key0 + 16 * u + 2 * cc + (t & 1) + 8 * (t >> 1) >= seq.len) {
#pragma unroll
                  for (int i = 0; i < D / 64; ++i) vr[u].w[t][i] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
          }
        }
        // running maximum
        bool up = false;
        float top[NR][2];
#pragma unroll
        for (int y = 0; y < NR; ++y)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = fmaxf(s[y][0][e], s[y][0][2 + e]);
#pragma unroll
            for (int u = 1; u < kBlocks; ++u) t = fmax3(t, s[y][u][e], s[y][u][2 + e]);
            top[y][e] = t * in.scale_log2;
            up = up || top[y][e] > m[y][e] + 8.f;
          }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int y = 0; y < NR; ++y)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float t = top[y][e];
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
              t = fmaxf(t, m[y][e]);
              const float f = t == m[y][e] ? 1.f : ex2(m[y][e] - t);
              m[y][e] = t;
              l[y][e] *= f;
              vsum[y][e] *= f;
#pragma unroll
              for (int j = 0; j < kTiles; ++j) acc[y][j][e] *= f, acc[y][j][2 + e] *= f;
            }
        }
        // weights, and O^T += V^T P^T
#pragma unroll
        for (int u = 0; u < kBlocks; ++u) {
          uint32_t pf[NR][2];
#pragma unroll
          for (int y = 0; y < NR; ++y)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              float w[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                w[e] = ex2(fmaf(s[y][u][2 * t + e], in.scale_log2, -base_of(m[y][e])));
                l[y][e] += w[e];
              }
              if constexpr (Q4) {
                const float2 pr = q4_pair(vr[u].pair[t]);
                const float mid = fmaf(8.f, pr.x, pr.y);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  vsum[y][e] = fmaf(w[e], mid, vsum[y][e]);
                  w[e] *= pr.x;
                }
              }
              const uint32_t pk = pack_bf16(w[0], w[1]);
              if constexpr (!Q4) {
                vsum[y][0] += __uint_as_float(pk << 16);
                vsum[y][1] += __uint_as_float(pk & 0xffff0000u);
              }
              pf[y][t] = transpose8x8(pk);
            }
          if constexpr (Q4) {
#pragma unroll
            for (int w = 0; w < D / 64; ++w)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint32_t lo = __byte_perm(vr[u].w[0][w], vr[u].w[1][w], q ? 0x7632 : 0x5410);
                const uint32_t hi = __byte_perm(vr[u].w[2][w], vr[u].w[3][w], q ? 0x7632 : 0x5410);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const int j = 4 * w + 2 * q + z;
                  const uint32_t a0 = codes_bf16(lo >> (8 * z)), a1 = codes_bf16(lo >> (8 * z + 4));
                  const uint32_t a2 = codes_bf16(hi >> (8 * z)), a3 = codes_bf16(hi >> (8 * z + 4));
#pragma unroll
                  for (int y = 0; y < NR; ++y) mma16816(acc[y][j], a0, a1, a2, a3, pf[y][0], pf[y][1]);
                }
              }
          } else {
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
              // the two channels of the tile's rows r and r + 8
              constexpr int kHiAt = D == 128 ? 0 : 4;
              const int e0 = j, e1 = j + kHiAt;
              auto word = [&](int t, int block, int e) -> uint32_t {
                const uint4& v = vr[u].w[t][block];
                return e / 2 == 0 ? v.x : e / 2 == 1 ? v.y : e / 2 == 2 ? v.z : v.w;
              };
              constexpr int kHiBlock = D == 128 ? 1 : 0;
              const uint32_t a0 = __byte_perm(word(0, 0, e0), word(1, 0, e0), e0 % 2 ? 0x7632 : 0x5410);
              const uint32_t a1 = __byte_perm(word(0, kHiBlock, e1), word(1, kHiBlock, e1), e1 % 2 ? 0x7632 : 0x5410);
              const uint32_t a2 = __byte_perm(word(2, 0, e0), word(3, 0, e0), e0 % 2 ? 0x7632 : 0x5410);
              const uint32_t a3 = __byte_perm(word(2, kHiBlock, e1), word(3, kHiBlock, e1), e1 % 2 ? 0x7632 : 0x5410);
#pragma unroll
              for (int y = 0; y < NR; ++y) mma16816(acc[y][j], a0, a1, a2, a3, pf[y][0], pf[y][1]);
            }
          }
        }
        if (more) {
#pragma unroll
          for (int u = 0; u < kBlocks; ++u) load_values(vr[u], v_base + (size_t)rows[u] * kRowBytes, vs_base + (size_t)rows[u] * 4);
        }
      }
    }

    // ---------------------------------------------------------- the warps' sums, joined
#pragma unroll
    for (int y = 0; y < NR; ++y)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          l[y][e] += __shfl_xor_sync(0xffffffffu, l[y][e], off);
          vsum[y][e] += __shfl_xor_sync(0xffffffffu, vsum[y][e], off);
        }
        const int row = y * 8 + 2 * cc + e;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          const float add = Q4 ? vsum[y][e] : 0.f;
          sh.o[warp][row][channel_of<D, Q4>(j, false, r)] = acc[y][j][e] + add;
          sh.o[warp][row][channel_of<D, Q4>(j, true, r)] = acc[y][j][2 + e] + add;
        }
        if (r == 0) {
          sh.m[warp][row] = m[y][e];
          sh.l[warp][row] = l[y][e];
          sh.div[warp][row] = Q4 ? l[y][e] : vsum[y][e];
        }
      }
    __syncthreads();
    // four channels of a row a thread; rows of no token are left out
    const int rows_here = min(kRows, seq.n * in.g - rb * kRows);
    float* part = in.partial + (size_t)slot * kRows * kPartial<D>;
    for (int i = threadIdx.x; i < rows_here * (D / 4); i += kThreads) {
      const int row = i / (D / 4), d = 4 * (i % (D / 4));
      float mm = sh.m[0][row];
#pragma unroll
      for (int w = 1; w < kW; ++w) mm = fmaxf(mm, sh.m[w][row]);
      float ll = 0.f, div = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        if (sh.l[w][row] == 0.f) continue;  // saw no key
        const float f = ex2(sh.m[w][row] - base_of(mm));
        const float4 v = *reinterpret_cast<const float4*>(&sh.o[w][row][d]);
        ll += sh.l[w][row] * f;
        div += sh.div[w][row] * f;
        o.x += v.x * f, o.y += v.y * f, o.z += v.z * f, o.w += v.w * f;
      }
      if (in.cluster > 1) {
        *reinterpret_cast<float4*>(&sh.o[0][row][d]) = o;
        if (d == 0) sh.all[row] = make_float4(mm, ll, div, 0.f);
      } else if (slot < 0) {
        const int at = rb * kRows + row;
        const size_t out = (size_t)(seq.first + at / in.g) * in.heads + h * in.g + at % in.g;
        const float inv = row_scale(ll, div, seq.len - seq.n + at / in.g);
        *reinterpret_cast<uint2*>(in.o + out * D + d) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (in.lse && d == 0) in.lse[out] = row_lse(mm, ll);
      } else {
        *reinterpret_cast<float4*>(part + row * kPartial<D> + d) = o;
        if (d == 0) *reinterpret_cast<float4*>(part + row * kPartial<D> + D) = make_float4(mm, ll, div, 0.f);
      }
    }
    __syncthreads();
    // ---------------------------------------------------------- and the cluster's CTAs', each a part of the rows
    if (in.cluster > 1) {
      cluster_sync();
      for (int i = rank * kThreads + threadIdx.x; i < rows_here * (D / 4); i += in.cluster * kThreads) {
        const int row = i / (D / 4), d = 4 * (i % (D / 4));
        float4 ml[kMaxCluster], v[kMaxCluster];
#pragma unroll
        for (int p = 0; p < kMaxCluster; ++p) {
          ml[p] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
          v[p] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (p < in.cluster) ml[p] = ld_cluster16(&sh.all[row], p), v[p] = ld_cluster16(&sh.o[0][row][d], p);
        }
        float mm = -INFINITY, ll = 0.f, div = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int p = 0; p < kMaxCluster; ++p) mm = fmaxf(mm, ml[p].x);
#pragma unroll
        for (int p = 0; p < kMaxCluster; ++p) {
          const float f = ex2(ml[p].x - base_of(mm));
          ll = fmaf(ml[p].y, f, ll);
          div = fmaf(ml[p].z, f, div);
          o.x = fmaf(v[p].x, f, o.x), o.y = fmaf(v[p].y, f, o.y);
          o.z = fmaf(v[p].z, f, o.z), o.w = fmaf(v[p].w, f, o.w);
        }
        const int at = rb * kRows + row;
        const size_t out = (size_t)(seq.first + at / in.g) * in.heads + h * in.g + at % in.g;
        const float inv = row_scale(ll, div, seq.len - seq.n + at / in.g);
        *reinterpret_cast<uint2*>(in.o + out * D + d) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (in.lse && d == 0) in.lse[out] = row_lse(mm, ll);
      }
      cluster_sync();  // nobody leaves while its sums are being read
    }
  }
}

// Joins the partial sums of units that the line's cuts run through.  CTA i
// stands for cut i + 1; the CTAs of one unit's cuts share its rows out.  They
// find the unit by themselves, while the sums are still being made.
template <int D, bool Q4, int NR>
__global__ void __launch_bounds__(kJoinThreads) s2_cache_join_kernel(const __grid_constant__ CacheArgs c,
                                                                     const __grid_constant__ AttnIn in) {
  constexpr int kStep = 16 * step_blocks<Q4>();
  constexpr int kRows = 8 * NR;
  __shared__ long long line_sh[kJoinThreads / 32 + 2];
  __shared__ JoinShared<D> sh;
  auto weight = [&](int i) { return seq_steps<NR>(c, in, i, kStep, true); };
  int b;
  long long seq_first;
  const Line line =
      find_piece<kJoinThreads>(c.B, in.pieces, in.min_piece, blockIdx.x + 1, line_sh, weight, b, seq_first);
  const long long cut = line.piece * (blockIdx.x + 1);
  JoinCut u;
  u.rows = 0;
  if (cut < line.total) {
    const Seq seq = load_seq(c, b);
    const int steps = steps_of(seq.len, kStep), blocks = row_blocks<NR>(seq.n, in.g), span = steps + kUnitSteps;
    const long long unit = quotient(cut - seq_first, span);
    const long long first = seq_first + unit * span + kUnitSteps;  // of its steps
    if (cut > first) {  // and not before the unit's first step
      const int h = (int)quotient(unit, blocks), rb = (int)(unit - (long long)h * blocks);
      u.rows = min(kRows, seq.n * in.g - rb * kRows);
      u.begin = u.p0 = (int)quotient(first, line.piece);
      u.p1 = (int)quotient(first + steps - 1, line.piece);
      u.nth = (int)blockIdx.x - u.p0;
      u.helpers = u.p1 - u.p0;
      u.tok = seq.first;
      u.place = seq.len - seq.n;
      u.row0 = rb * kRows;
      u.head = h * in.g;
    }
  }
  // every CTA waits, also one with nothing to do: the stream's next launch counts on this one's end alone
  asm volatile("griddepcontrol.wait;" ::: "memory");
  join_rows<D>(sh, u, in.partial, kRows, in.g, in.heads, in.o, in.lse);
}

// CTAs to a whole unit, so that few units fill the GPU: as many as are resident at once, up to 8, with 64 keys each at
// least (32 units of 200 keys in bf16: 1 to 8 CTAs 7.0, 7.2, 6.3, 6.8 us).
static int cluster_of(int64_t units, int64_t max_len, int resident) {
  int cs = 1;
  while (2 * cs <= kMaxCluster && 2 * cs * units <= resident && max_len >= 64 * 2 * cs) cs *= 2;
  return cs;
}

// Whether units are cut and joined in a second launch, or whole ones taken by clusters.  The latter needs one launch and
// no partial sums in memory, but the longest unit sets its time, and only a bound of the lengths is known.  The limits, 256
// keys a CTA of a cluster of four or eight and 512 keys for one or two CTAs, are where it is about as fast as the former
// with lengths of half the bound on the average (us whole and cut.  Clusters: 32 units of 513 keys 7.6 and 9.5, of 1024 8.0
// and 9.7, of 2048 9.9 and 12.8, of 4096 14.1 and 16.2; 8 units of 2048 8.6 and 8.7, of 4096 11.3 and 9.8; 128 units, two
// CTAs each, of 513 10.7 and 13.4, of 2048 25.3 and 25.4.  One CTA each, keys spread over 1 to 512: 512 units 18.0 and
// 19.6, 1024 30.1 and 32.3, 2048 58.0 and 55.1, in 4 bits 13.5 and 17.7, 22.1 and 25.8, 42.0 and 41.7; over 1 to 1024, 512
// units 31.5 and 29.0; all of 512, 512 units 32.0 and 28.4, in 4 bits 14.9 and 21.5).
static bool cut_units(int64_t max_len, int cluster) {
  return max_len == 0 || max_len > 256 * (cluster > 2 ? cluster : 2);
}

template <int D, bool Q4, int NR>
static int decode_impl(const CacheArgs& c, const AttnIn& in0, int64_t max_len, cudaStream_t stream) {
  AttnIn in = in0;
  // units at most: every sequence rounds its rows up to blocks
  const int64_t rows = (int64_t)c.T * in.g / (8 * NR) + (c.T < c.B ? c.T : c.B);
  const int64_t units = c.heads * (c.starts ? rows : (int64_t)c.B * ((in.g + 8 * NR - 1) / (8 * NR)));
  constexpr int kResident = 148 * ctas_per_sm<Q4, NR>();
  in.cluster = cluster_of(units, max_len, kResident);
  const bool cut = cut_units(max_len, in.cluster);
  if (cut) in.cluster = 1;
  in.pieces = cut ? kResident : 0;
  in.min_piece = cut ? kUnitSteps + kW : 1;  // a step for each warp
  constexpr int kBytes = (int)sizeof(DecodeShared<D, NR>);
  cudaError_t e;
  if (kBytes > 48 * 1024) {
    e = cudaFuncSetAttribute(s2_cache_decode_kernel<D, Q4, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return (int)e;
  }
  if (!cut && units >= (int64_t(1) << 31)) return (int)cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  cfg.stream = stream;
  cfg.attrs = at;
  if (in.cluster > 1) {
    cfg.gridDim = dim3((unsigned)(units * in.cluster));
    cfg.blockDim = dim3(kW * 32);
    cfg.dynamicSmemBytes = kBytes;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)in.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, s2_cache_decode_kernel<D, Q4, NR>, c, in);
  }
  s2_cache_decode_kernel<D, Q4, NR><<<(unsigned)(cut ? in.pieces : units), kW * 32, kBytes, stream>>>(c, in);
  e = cudaGetLastError();
  if (e != cudaSuccess || !cut) return (int)e;
  cfg.gridDim = dim3(in.pieces - 1);
  cfg.blockDim = dim3(kJoinThreads);
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, s2_cache_join_kernel<D, Q4, NR>, c, in);
}

template <int D, bool Q4>
static int decode_rows(const CacheArgs& c, const AttnIn& in, int64_t rows, int64_t max_len, cudaStream_t stream) {
  return rows <= 8 ? decode_impl<D, Q4, 1>(c, in, max_len, stream) : decode_impl<D, Q4, 2>(c, in, max_len, stream);
}

int launch_cache_decode(const CacheArgs& c, const AttnIn& in, int D, bool q4, int64_t rows, int64_t max_len,
                        cudaStream_t stream) {
  if (D == 64)
    return q4 ? decode_rows<64, true>(c, in, rows, max_len, stream) : decode_rows<64, false>(c, in, rows, max_len, stream);
  return q4 ? decode_rows<128, true>(c, in, rows, max_len, stream) : decode_rows<128, false>(c, in, rows, max_len, stream);
}

size_t cache_decode_partial_bytes(int D) { return (size_t)2 * kDecodePieces * 16 * (D + 4) * sizeof(float); }

}  // namespace s2
