// s2_cache_chunk.cu -- attention of many new tokens over a paged cache
// (chunks of prompts): the operator of s2_cache_attn.cu where the products
// bound it, on the tensor cores (tcgen05, TMEM), fed by TMA.
//
// Rows: the g query heads of a key/value head share its keys, so a tile of
// query rows is (128 / g tokens) x (g heads), 128 rows for g a power of two, and
// a unit is two such tiles (A, B: consecutive tokens) of one key/value head.
// Its keys go by in tiles of 128: 128 / S pages, each brought by TMA into its
// rows of the tile (or, in 4 bits, unpacked there by two warps).
//
// Work: the units' keys form one line (s2_cache.cuh) cut into one piece per
// SM, so a few long units load all SMs as well as many short ones.  CTAs stay
// for their whole piece: tensor memory, barriers and the load pipeline run on
// from unit to unit, so a unit's epilogue overlaps the next one's first
// products.  A unit cut by a border leaves partial sums for
// s2_cache_chunk_join.
//
// Warp roles: warps 0-3 softmax of tile A (thread = query row = TMEM lane),
// 4-7 of tile B, 8 TMA, 9 MMA issue; with 4-bit pages warps 10 and 11
// unpack (with or without them the softmax warps have 168 registers).  MMA
// order, TMEM layout and the softmax are those of s2_fwd.cu: S and P share columns, P feeds O += P V
// from TMEM, and the running maximum moves when a score passes it by more than 8 (in powers of two).
//
// 4 bits: packed rows come by bulk copies and are unpacked to whole numbers
// that bf16 holds as they are, 128 + code for keys (no subtraction) and code - 8
// for values (so that rounded weights meet small numbers).  The softmax applies
// scale and min of each key: s = sk (q·k') + (mk - 128 sk) sum(q) (2^-5 of it, s2_cache.cuh); the weight that
// goes into the product is p·sv (rounded once to bf16, relative 2^-8), and
// sum p (mv + 8 sv), the same for every channel, is kept beside O.
//
// Weights are rounded to bf16 for the product (2^-8 of each at most), and O is
// divided by their sum in 32 bits as it was before that rounding: with the sum of the rounded
// ones, as s2_cache_attn.cu has it for bf16 rows, o's error against 64 bits is 0.00199
// of its norm and not 0.00204, but 2048 tokens over 16384 keys take 464 us and
// not 442, since the softmax warps set the pace.
//
// Measured: 2048 tokens (32 heads, 8 key heads, D 128) over 16384 keys 434
// to 457 us on several GPUs in a captured graph, 1130 to 1190 TFLOP/s (the products alone would
// take 312), and 502 to 520 (about 1010) called one by one, when the power cap
// holds the clock down: the softmax's hand-off chain bounds it (tensor pipe 55%).  4 bits,
// three chunks of 260 to 1000 tokens over 3000 to 12000 keys 336 us, where no
// pipe is near its limit (issue 45%, tensor and XU 34%): it is the softmax warps' work on
// each key's scale and min that is long.  Short calls: 60 tokens over 8000 keys 33 us, of which
// finding the first segment takes 4, loading 2, the sums' way out 3, the join 10.
#include <climits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "s2_cache.cuh"
#include "s2_cache_join.cuh"
#include "s2_kernels.h"
#include "sm100_ptx.cuh"

namespace s2 {

namespace chunk {

constexpr int kT = 128;  // rows of a tile, of queries and of keys
constexpr int kChunkBytes = kT * 128;
constexpr int kSegs = 48;          // units (or parts) that a CTA looks ahead
constexpr int kScaleSlots = 2;
constexpr int kRawSlots = 3;       // key tiles of packed rows in flight (4-bit pages)
constexpr long long kUnitKeys = 256;  // what starting and ending a unit costs, in keys

template <bool Q4>
__host__ __device__ constexpr int threads() { return Q4 ? 384 : 320; }
template <bool Q4>
__host__ __device__ constexpr int slots() { return Q4 ? 3 : 5; }

enum Bar {
  KV_FULL = 0,                          // + slot (5)
  KV_EMPTY = 5,                         // + slot (5)
  S_FULL = 10,                          // + tile (2)
  P_FULL = 12,                          // + tile (2)
  O_FULL = 14,                          // + tile (2)
  Q_FULL = 16,
  Q_EMPTY = 17,
  TAIL = 18,                            // the last value tile of a sequence, before its unused rows are zeroed
  MMA_DONE = 19,
  SC_FULL = 20,                         // + scale slot (2)
  SC_EMPTY = 22,                        // + scale slot (2)
  RAW_FULL = 24,                        // + raw slot (3)
  RAW_EMPTY = 27,                       // + raw slot (3)
  NUM_BARS = 30
};

// Part of a unit that a CTA computes.
struct Seg {
  int b, h;
  int tok;     // first new token of tile A on the packed axis
  int left;    // new tokens of the sequence from there on
  int place;   // place of that token
  int len;
  int t0, t1;  // key tiles
  int slot;    // partial sums' slot, or -1: the unit is whole and its rows are final
};

// Where a CTA's walk along the line stands.
struct Walk {
  long long at, x0, x1;  // of the piece [x0, x1)
  long long start;       // where sequence b begins
  long long piece;
  int b, h, j;
};

template <int D, bool Q4>
struct Layout {
  static constexpr int kQBytes = kT * D * 2;
  static constexpr int kKVBytes = kT * D * 2;
  static constexpr int kQ = 0;
  static constexpr int kKV = 2 * kQBytes;
  static constexpr int kScale = kKV + slots<Q4>() * kKVBytes;  // per slot {s, s, m, m} of each two keys, then the same of the values
  // packed rows of a key tile: key codes, value codes, key pairs, value pairs
  static constexpr int kRaw = kScale + (Q4 ? kScaleSlots * kT * 16 : 0);
  static constexpr int kRawBytes = kT * (D + 8);
  static constexpr int kBars = kRaw + (Q4 ? kRawSlots * kRawBytes : 0);
  static constexpr int kMisc = kBars + NUM_BARS * 8;
  static constexpr int kLine = kMisc + 16;  // make_line's and find_seq's sums
  static constexpr int kWalk = kLine + 18 * 8;
  static constexpr int kSeg = kWalk + (int)sizeof(Walk);
  static constexpr int kBytes = kSeg + (int)sizeof(Seg) * (Q4 ? kSegs : 16);
  static constexpr int kAlloc = kBytes + 1024;
};

// Sequence b cut into units: pair j holds new tokens [j·d, (j + 1)·d), d = 2·(128 / g), which see up to
// first + (j + 1)·d keys.  A unit weighs as many keys and kUnitKeys; sums of weights have a closed form.  (That
// the weights are exact, and a piece at least 384, leaves a key tile in every piece between a unit's first and last.)
struct Units {
  long long first;  // place of the first new token; negative where a sequence is shorter than its new tokens
  int n, d, pairs;
  int blind;        // pairs that see no key
  __device__ __forceinline__ Units(const Seq& s, int per_tile) {
    n = s.n;
    d = 2 * per_tile;
    pairs = (n + d - 1) / d;
    first = (long long)s.len - s.n;
    blind = first < 0 ? (s.n - s.len) / d : 0;
  }
  __device__ __forceinline__ long long weight(int j) const {
    return kUnitKeys + (j == pairs - 1 ? first + n : j < blind ? 0 : first + (long long)(j + 1) * d);
  }
  __device__ __forceinline__ long long before(int j) const {
    const long long see = j > blind ? j - blind : 0;  // pairs before j that see keys: blind .. j - 1
    return j * kUnitKeys + see * first + (long long)d * (see * (blind + 1) + see * (see - 1) / 2);
  }
  __device__ __forceinline__ long long head() const { return before(pairs - 1) + kUnitKeys + first + n; }
  // The pair that holds point r of a head's units.
  __device__ __forceinline__ int find(long long r) const {
    int lo = 0, hi = pairs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (before(mid) <= r) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
};

// Last key tile that `count` tokens from place `place` on see, or -1.
__device__ __forceinline__ int last_tile(int place, int count) {
  const int p = place + count - 1;
  return count > 0 && p >= 0 ? p / kT : -1;
}
// Key tiles of pair j of a sequence.
__device__ __forceinline__ int pair_tiles(const Seq& s, const Units& u, int j) {
  const int first = j * u.d;
  return last_tile(s.len - s.n + first, min(u.d, s.n - first)) + 1;
}
// Key tiles of a unit that lie before point w of its weight (the same for all that ask, and growing with w).  Where in
// the unit a cut falls need not be exact: 32 bits are off by 2^-22 of the unit at most, far less than a piece.
__device__ __forceinline__ int tile_at(int tiles, long long w, long long weight) {
  if (w >= weight) return tiles;
  return min(tiles, __float2int_rd(__fdiv_rn(__fmul_rn((float)(int)w, (float)tiles), (float)(int)weight)));
}

// The next segments of a CTA's piece (one thread); returns their number.  What the piece's end cuts goes to `cut`.
__device__ __noinline__ int walk_on(Walk& w, const CacheArgs& c, int g_heads, int per_tile, Seg* segs, int most,
                                    JoinCut* cut) {
  int k = 0;
  if (w.at >= w.x1) return 0;
  Seq s = load_seq(c, w.b);
  while (k < most && w.at < w.x1) {
    const Units units(s, per_tile);
    const int u_d = units.d;
    if (w.j >= units.pairs) {
      w.j = 0;
      ++w.h;
    }
    if (s.n == 0 || w.h >= c.heads) {
      if (s.n > 0) w.start += units.head() * c.heads;
      w.h = w.j = 0;
      s = load_seq(c, ++w.b);
      continue;
    }
    const long long weight = units.weight(w.j);
    const long long begin = w.start + w.h * units.head() + units.before(w.j), end = begin + weight;
    const int tiles = pair_tiles(s, units, w.j);
    const int ta = tile_at(tiles, max(w.at, begin) - begin, weight);
    const int tb = tile_at(tiles, min(w.x1, end) - begin, weight);
    if (tiles ? tb > ta : w.at <= begin) {
      Seg& g = segs[k++];
      g.b = w.b;
      g.h = w.h;
      g.tok = s.first + w.j * u_d;
      g.left = s.n - w.j * u_d;
      g.place = s.len - s.n + w.j * u_d;
      g.len = s.len;
      g.t0 = ta;
      g.t1 = tb;
      g.slot = (ta == 0 && tb == tiles) ? -1 : 2 * (int)blockIdx.x + (begin < w.x0 ? 0 : 1);
    }
    if (end > w.x1 && tiles > 0) {
      const int p0 = (int)quotient(begin, w.piece), p1 = (int)quotient(end - 1, w.piece);
      JoinCut u;
      u.rows = min(s.n - w.j * u_d, u_d) * g_heads;
      u.nth = (int)blockIdx.x - p0;
      u.helpers = p1 - p0;
      u.begin = p0;
      // pieces between hold tiles; the first and the last may hold none
      u.p0 = p0 + (tile_at(tiles, w.piece * (p0 + 1) - begin, weight) == 0);
      u.p1 = p1 - (tile_at(tiles, w.piece * p1 - begin, weight) == tiles);
      u.tok = s.first + w.j * u_d;
      u.place = s.len - s.n + w.j * u_d;
      u.row0 = 0;
      u.head = w.h * g_heads;
      if (u.p0 < u.p1) *cut = u;  // else one piece has all of the unit's tiles, and writes its rows
    }
    w.at = min(w.x1, end);
    ++w.j;
  }
  return k;
}

// {scale, scale, min, min} of four times two keys, the same for all lanes: four loads at once, so that their wait is shared.
// The clobber keeps them where they stand: moved up together they would fill the registers.
struct Pairs8 {
  float4 p[4];
};
__device__ __forceinline__ void load_pairs(Pairs8& v, uint32_t at) {
  asm volatile(
      "ld.shared.v4.f32 {%0,%1,%2,%3}, [%16];\n\t"
      "ld.shared.v4.f32 {%4,%5,%6,%7}, [%16+16];\n\t"
      "ld.shared.v4.f32 {%8,%9,%10,%11}, [%16+32];\n\t"
      "ld.shared.v4.f32 {%12,%13,%14,%15}, [%16+48];"
      : "=f"(v.p[0].x), "=f"(v.p[0].y), "=f"(v.p[0].z), "=f"(v.p[0].w), "=f"(v.p[1].x), "=f"(v.p[1].y),
        "=f"(v.p[1].z), "=f"(v.p[1].w), "=f"(v.p[2].x), "=f"(v.p[2].y), "=f"(v.p[2].z), "=f"(v.p[2].w),
        "=f"(v.p[3].x), "=f"(v.p[3].y), "=f"(v.p[3].z), "=f"(v.p[3].w)
      : "r"(at)
      : "memory");
}

// Partial sums lie as float4 [slot][query tile][channels / 4, then maximum, sum, divisor][row]: a warp's 32 rows write
// and read 512 bytes side by side.  (Row by row, the 32 lines of each store took 5 us a segment.)
template <int D>
__device__ __forceinline__ size_t partial_at(int slot, int x, int c4) {
  return (((size_t)slot * 2 + x) * (D / 4 + 1) + c4) * kT;
}

// Lanes 4k .. 4k + 3 hold four 16-byte pieces each of their rows: afterwards lane 4k + i holds piece i of the four rows.
__device__ __forceinline__ void transpose_pieces(uint32_t (&w)[4][4], int lane) {
#pragma unroll
  for (int bit = 1; bit < 4; bit *= 2) {
    const bool up = lane & bit;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a & bit) continue;
      const int b = a | bit;
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[a][z] : w[b][z], bit);
        if (up)
          w[a][z] = got;
        else
          w[b][z] = got;
      }
    }
  }
}

}  // namespace chunk

template <int D, bool Q4>
__global__ void __launch_bounds__(chunk::threads<Q4>(), 1)
    s2_cache_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CacheArgs c,
                          const __grid_constant__ AttnIn in) {
  using namespace chunk;
  using L = Layout<D, Q4>;
  constexpr int kThreads = threads<Q4>();
  constexpr int kSlots = slots<Q4>();
  constexpr int kChunks = D / 64;
  constexpr int kList = Q4 ? kSegs : 16;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 256) {  // the TMA warp
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* count = reinterpret_cast<volatile int*>(tmem_slot + 2);
  long long* line_sh = reinterpret_cast<long long*>(smem + L::kLine);
  Walk* walk = reinterpret_cast<Walk*>(smem + L::kWalk);
  Seg* segs = reinterpret_cast<Seg*>(smem + L::kSeg);
  int* const status = c.status;
  const uint32_t sbar = sb + L::kBars;
#define bar(i) (sbar + 8u * (uint32_t)(i))
#define sQ(x) (sb + L::kQ + (uint32_t)(x) * L::kQBytes)
#define sKV(slot) (sb + L::kKV + (uint32_t)(slot) * L::kKVBytes)

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int per_tile = kT / in.g;  // tokens of a query tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar(KV_FULL + i), Q4 ? 64 : 1);
      mbar_init(bar(KV_EMPTY + i), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(S_FULL + x), 1);
      mbar_init(bar(P_FULL + x), 128);
      mbar_init(bar(O_FULL + x), 1);
    }
    mbar_init(bar(Q_FULL), 1);
    mbar_init(bar(Q_EMPTY), Q4 ? 1 + 256 : 1);
    mbar_init(bar(TAIL), 1);
    mbar_init(bar(MMA_DONE), 1);
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(bar(SC_FULL + i), 64);
      mbar_init(bar(SC_EMPTY + i), 256);
    }
    for (int i = 0; i < kRawSlots; ++i) {
      mbar_init(bar(RAW_FULL + i), 1);
      mbar_init(bar(RAW_EMPTY + i), 64);
    }
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // The CTA's piece of the line, and the sequence that it begins in.
  auto weight_of = [&](int b) -> long long {
    const Seq s = load_seq(c, b);
    return s.n > 0 ? Units(s, per_tile).head() * c.heads : 0;
  };
  int b_first;
  long long b_start;
  const Line line = find_piece<kThreads>(c.B, in.pieces, in.min_piece, blockIdx.x, line_sh, weight_of, b_first, b_start);
  const long long x0 = line.piece * blockIdx.x, x1 = min(x0 + line.piece, line.total);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Thread 0's walk along the line; its state is in shared memory, the registers are the softmax's.
  if (threadIdx.x == 0) {
    walk->b = walk->h = walk->j = 0;
    walk->at = x0;
    walk->x0 = x0;
    walk->x1 = max(x0, x1);
    walk->start = b_start;
    walk->piece = line.piece;
    static_cast<JoinCut*>(in.cuts)[blockIdx.x].rows = 0;
    if (x0 < x1) {
      const Units u(load_seq(c, b_first), per_tile);
      walk->b = b_first;
      walk->h = (int)quotient(x0 - b_start, u.head());
      walk->j = u.find(x0 - b_start - walk->h * u.head());
    }
  }

  // All roles walk the same list of segments; thread 0 writes it, in pieces.  Counters of barrier phases run on
  // from segment to segment, and each role keeps its own, so that the softmax's registers hold nothing else's.
  bool ok = true;
  auto next_list = [&]() -> int {
    __syncthreads();  // everyone is done with the last list
    if (threadIdx.x == 0) *count = *abort_flag ? 0 : walk_on(*walk, c, in.g, per_tile, segs, kList,
                                                            static_cast<JoinCut*>(in.cuts) + blockIdx.x);
    __syncthreads();
    return *count;
  };
#define FOR_SEGMENTS                                        \
  for (int k_segs = next_list(); k_segs > 0; k_segs = next_list()) \
    for (int si = 0; si < k_segs && ok; ++si)
// Tokens of the segment's two query tiles, the last key tile of each (or -1), and whether they have keys here.
#define SEGMENT_OF(g)                                                                   \
  const int cntA = min(g.left, per_tile), cntB = min(g.left - per_tile, per_tile);      \
  const int lastA = min(last_tile(g.place, cntA), g.t1 - 1);                            \
  const int lastB = min(last_tile(g.place + per_tile, cntB), g.t1 - 1);                 \
  const bool hasA = lastA >= g.t0, hasB = lastB >= g.t0, keys = g.t1 > g.t0;

  if (warp == 8) {
    // ------------------------------------------------------------ TMA
    int e = 0;       // key and value tiles so far: the e-th goes to slot e % kSlots
    int n_seg = 0;   // segments with keys
    int n_tail = 0;
    int n_raw = 0;   // key tiles of packed rows
    FOR_SEGMENTS {
      const Seg g = segs[si];
      SEGMENT_OF(g)
      if (!keys) continue;
      if (lane == 0) {
        if (n_seg > 0) ok = s2_wait(bar(Q_EMPTY), (n_seg - 1) & 1, abort_flag, status, 1);
        if (ok) {
          const uint32_t bytes = (uint32_t)(per_tile * in.g) * 128 * kChunks;
          mbar_arrive_expect_tx(bar(Q_FULL), (hasA ? bytes : 0) + (hasB ? bytes : 0));
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (x ? hasB : hasA)
              for (int ch = 0; ch < kChunks; ++ch)
                tma_load_3d(sQ(x) + ch * kChunkBytes, &tmQ, ch * 64, g.h * in.g, g.tok + x * per_tile, bar(Q_FULL));
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++n_seg;
      if constexpr (Q4) {
        // a page's packed rows of one head are contiguous: a lane copies one of the tile's four parts of a page
        const int pages = kT >> c.log2s;
        for (int t = g.t0; t < g.t1 && ok; ++t) {
          const int live = min(pages, ((g.len - t * kT - 1) >> c.log2s) + 1);
          const int part = lane / 8, i = lane % 8;  // pages <= 8
          int page = 0;
          if (i < live) page = page_of(c, g.b, t * kT + (i << c.log2s));
          const int slot = n_raw % kRawSlots;
          if (n_raw >= kRawSlots)
            ok = s2_wait(bar(RAW_EMPTY + slot), ((n_raw / kRawSlots) - 1) & 1, abort_flag, status, 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(RAW_FULL + slot), (uint32_t)(live << c.log2s) * (D + 8));
          __syncwarp();
          if (i < live) {
            const int bytes = part < 2 ? D / 2 : 4;  // of a row
            const void* from = part == 0 ? c.k : part == 1 ? c.v : part == 2 ? c.k_scale : c.v_scale;
            const uint32_t to = sb + L::kRaw + slot * L::kRawBytes + (part < 2 ? part * kT * (D / 2) : kT * D + (part - 2) * kT * 4);
            bulk_load(to + (i << c.log2s) * bytes,
                      static_cast<const uint8_t*>(from) + row_of(c, page, g.h, 0) * bytes,
                      (uint32_t)bytes << c.log2s, bar(RAW_FULL + slot));
          }
          ++n_raw;
        }
      } else {
        const int pages = kT >> c.log2s;  // of a tile
        for (int t = g.t0; t < g.t1 && ok; ++t) {
          const int live = min(pages, ((g.len - t * kT - 1) >> c.log2s) + 1);
          int page = 0;
          if (lane < live) page = page_of(c, g.b, t * kT + (lane << c.log2s));
          const bool tail = g.len - t * kT < kT;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int slot = e % kSlots;
            if (e >= kSlots) ok = s2_wait(bar(KV_EMPTY + slot), ((e / kSlots) - 1) & 1, abort_flag, status, 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t full = v && tail ? bar(TAIL) : bar(KV_FULL + slot);
            if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(live << c.log2s) * 128 * kChunks);
            __syncwarp();
            if (lane < live) {
              for (int ch = 0; ch < kChunks; ++ch)
                tma_load_3d(sKV(slot) + ch * kChunkBytes + ((lane << c.log2s) * 128), v ? &tmV : &tmK, ch * 64, 0,
                            page * c.heads + g.h, full);
            }
            if (v && tail) {
              // rows behind the sequence may hold anything, and 0 times a NaN is a NaN
              if (!s2_wait_drain(bar(TAIL), n_tail & 1, status, 1)) *abort_flag = 1;
              ++n_tail;
              const int used = g.len - t * kT;
              for (int i = used * 8 * kChunks + lane; i < kT * 8 * kChunks; i += 32) {
                const int row = i / (8 * kChunks), piece = i % (8 * kChunks);
                st_shared_v4(sKV(slot) + (piece / 8) * kChunkBytes + row * 128 + (piece % 8) * 16, 0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(KV_FULL + slot));
            }
            ++e;
          }
        }
      }
    }
    // copies in flight land before shared memory is released (also after an abort)
    if (lane == 0) {
      if constexpr (Q4) {
        for (int d = (n_raw > kRawSlots ? n_raw - kRawSlots : 0); d < n_raw; ++d)
          s2_wait_drain(bar(RAW_FULL + d % kRawSlots), (d / kRawSlots) & 1, status, 1);
      } else {
        for (int d = (e > kSlots ? e - kSlots : 0); d < e; ++d)
          s2_wait_drain(bar(KV_FULL + d % kSlots), (d / kSlots) & 1, status, 1);
      }
      if (n_seg > 0) s2_wait_drain(bar(Q_FULL), (n_seg - 1) & 1, status, 1);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA
    int e = 0, n_seg = 0;
    int nA = 0, nB = 0;  // key tiles of each query tile
    FOR_SEGMENTS {
      const Seg g = segs[si];
      SEGMENT_OF(g)
      if (lane == 0 && keys) {
        constexpr uint32_t idesc_qk = umma_idesc_bf16(128, 128, 0, 0);
        constexpr uint32_t idesc_pv = umma_idesc_bf16(128, D, 0, 1);
#define ISSUE_QK(x, slot)                                                                              \
do {                                                                                                 \
  const uint64_t a0_ = umma_desc_sw128(sQ(x), 16, 1024), b0_ = umma_desc_sw128(sKV(slot), 16, 1024); \
  _Pragma("unroll") for (int kk = 0; kk < D / 16; ++kk) {                                            \
    const uint64_t off_ = ((kk / 4) * kChunkBytes + (kk % 4) * 32) >> 4;                             \
    umma_ss(tmem + (x) * 128, a0_ + off_, b0_ + off_, idesc_qk, kk > 0);                             \
  }                                                                                                  \
} while (0)
#define ISSUE_PV(x, slot, acc)                                                                  \
do {                                                                                          \
  const uint64_t b0_ = umma_desc_sw128(sKV(slot), kChunkBytes, 1024);                         \
  _Pragma("unroll") for (int kk = 0; kk < kT / 16; ++kk) {                                    \
    umma_ts(tmem + 256 + (x) * D, tmem + (x) * 128 + 8 * kk, b0_ + (uint64_t)(kk * 2048 >> 4), \
            idesc_pv, ((acc) || kk > 0) ? 1u : 0u);                                           \
  }                                                                                           \
} while (0)
#define WAIT_KV(i) s2_wait(bar(KV_FULL + (i) % kSlots), ((i) / kSlots) & 1, abort_flag, status, 2)
        ok = s2_wait(bar(Q_FULL), n_seg & 1, abort_flag, status, 2);
        ++n_seg;
        int eK = e++;
        if (ok) ok = WAIT_KV(eK);
        if (ok) {
          if (hasA) {
            ISSUE_QK(0, eK % kSlots);
            umma_commit(bar(S_FULL + 0));
          }
          if (hasB) {
            ISSUE_QK(1, eK % kSlots);
            umma_commit(bar(S_FULL + 1));
          }
          umma_commit(bar(KV_EMPTY + eK % kSlots));
          if (g.t1 - g.t0 == 1) umma_commit(bar(Q_EMPTY));
        }
        for (int t = g.t0; t < g.t1 && ok; ++t) {
          const bool more = t + 1 < g.t1;
          const int eV = e++;
          eK = more ? e++ : 0;
          ok = WAIT_KV(eV);
          if (ok && more) ok = WAIT_KV(eK);
          if (!ok) break;
          const int sV = eV % kSlots, sK = eK % kSlots;
          if (t <= lastA) {
            ok = s2_wait(bar(P_FULL + 0), nA & 1, abort_flag, status, 2);
            if (!ok) break;
            tc_fence_after();
            ISSUE_PV(0, sV, t > g.t0);
            ++nA;
          }
          if (more && t + 1 <= lastA) {
            ISSUE_QK(0, sK);
            umma_commit(bar(S_FULL + 0));
          }
          if (t <= lastB) {
            ok = s2_wait(bar(P_FULL + 1), nB & 1, abort_flag, status, 2);
            if (!ok) break;
            tc_fence_after();
            ISSUE_PV(1, sV, t > g.t0);
            ++nB;
          }
          if (more && t + 1 <= lastB) {
            ISSUE_QK(1, sK);
            umma_commit(bar(S_FULL + 1));
          }
          umma_commit(bar(KV_EMPTY + sV));
          if (more) {
            umma_commit(bar(KV_EMPTY + sK));
            if (t + 2 == g.t1) umma_commit(bar(Q_EMPTY));
          }
        }
        if (ok && hasA) umma_commit(bar(O_FULL + 0));
        if (ok && hasB) umma_commit(bar(O_FULL + 1));
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    // every product is complete before tensor memory is released (also after an abort)
    if (lane == 0) {
      umma_commit(bar(MMA_DONE));
      s2_wait_drain(bar(MMA_DONE), 0, status, 2);
    }
    __syncwarp();
  } else if (Q4 && warp >= 10) {
    // ------------------------------------------------------------ unpacking of 4-bit pages
    int e = 0;
    int n_raw = 0, n_sc = 0;  // key tiles (raw slots, scale slots)
    FOR_SEGMENTS {
      const Seg g = segs[si];
      const bool keys = g.t1 > g.t0;
      // 16 bytes of a row at a time: channels [16i, 16i + 16) in the low halves, D/2 further in the high
      // ones.  A quarter of a warp reads 128 bytes in a row and writes 8 different banks' worth of pieces.
      if (!keys) continue;
      const int tid = threadIdx.x - 320;
      constexpr int kParts = D / 32;  // of a row
      auto unpack = [&](uint32_t raw, int slot, int used, bool centred) {
#pragma unroll 2
        for (int it = 0; it < 2 * kParts; ++it) {
          const int item = it * 64 + tid, row = item / kParts, i = item % kParts;
          uint32_t w[4];
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(raw + item * 16));
          // rows behind the sequence: zeros as values (their weight is 0 and 0 times anything must be 0)
          if (row >= used) w[0] = w[1] = w[2] = w[3] = 0x88888888u;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t o[8];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const uint32_t x = (w[z] >> (4 * half)) & 0x0f0f0f0fu;
              o[2 * z] = __byte_perm(x, 0x43u, 0x4140);  // 0x43, code: 128 + code in bf16
              o[2 * z + 1] = __byte_perm(x, 0x43u, 0x4342);
            }
            if (centred) {
#pragma unroll
              for (int z = 0; z < 8; ++z) o[z] = less_136(o[z]);
            }
            const int ch = half * (D / 2) + 16 * i, piece = (ch % 64) / 8;
            const uint32_t to = sKV(slot) + (ch / 64) * kChunkBytes + row * 128;
            st_shared_v4(to + ((piece ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
            st_shared_v4(to + (((piece + 1) ^ (row & 7)) << 4), o[4], o[5], o[6], o[7]);
          }
        }
      };
      auto claim = [&]() -> int {  // the next tile's slot, once its products are done
        const int slot = e % kSlots;
        if (e >= kSlots) ok = s2_wait(bar(KV_EMPTY + slot), ((e / kSlots) - 1) & 1, abort_flag, status, 8);
        ++e;
        return slot;
      };
      for (int t = g.t0; t < g.t1; ++t) {
        const int rs = n_raw % kRawSlots, sc = n_sc % kScaleSlots, used = g.len - t * kT;
        const uint32_t raw = sb + L::kRaw + rs * L::kRawBytes;
        ok = s2_wait(bar(RAW_FULL + rs), (n_raw / kRawSlots) & 1, abort_flag, status, 8);
        if (!ok) break;
        const int sK = claim();
        if (!ok) break;
        unpack(raw, sK, kT, false);  // rows behind the sequence are masked as keys
        fence_proxy_async_smem();
        mbar_arrive(bar(KV_FULL + sK));
        if (n_sc >= kScaleSlots)
          ok = s2_wait(bar(SC_EMPTY + sc), ((n_sc / kScaleSlots) - 1) & 1, abort_flag, status, 8);
        if (!ok) break;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int row = tid + 64 * y;
          const uint32_t* pairs = reinterpret_cast<const uint32_t*>(smem + L::kRaw + rs * L::kRawBytes + kT * D);
          const float2 k2 = q4_key(q4_pair(row < used ? pairs[row] : 0u)), v2 = q4_pair(row < used ? pairs[kT + row] : 0u);
          // {scale, scale, min, min} of two keys: adjacent registers for the softmax's packed arithmetic
          float* to = reinterpret_cast<float*>(smem + L::kScale) + sc * 4 * kT + (row / 2) * 4 + row % 2;
          to[0] = k2.x;
          to[2] = k2.y;  // codes come as 128 + code,
          to[2 * kT] = v2.x;
          to[2 * kT + 2] = fmaf(8.f, v2.x, v2.y);  // and as code - 8
        }
        mbar_arrive(bar(SC_FULL + sc));
        ++n_sc;
        const int sV = claim();
        if (!ok) break;
        unpack(raw + kT * (D / 2), sV, used, true);
        fence_proxy_async_smem();
        mbar_arrive(bar(KV_FULL + sV));
        mbar_arrive(bar(RAW_EMPTY + rs));
        ++n_raw;
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int x = warp / 4, wq = warp % 4;
    const int r = wq * 32 + lane;  // row of the tile == TMEM lane
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + x * 128;
    const uint32_t tO = tmem + lane_off + 256 + x * D;
    const int tok = r / in.g;  // of the tile
    int nS = 0, nO = 0;        // key tiles, and segments with keys, of this query tile
    int n_seg = 0, n_sc = 0;
    FOR_SEGMENTS {
      const Seg& g = segs[si];
      const bool keys = g.t1 > g.t0;
      const int cnt = x ? min(g.left - per_tile, per_tile) : min(g.left, per_tile);
      const int last = min(last_tile(g.place + x * per_tile, cnt), g.t1 - 1);
      const bool has = last >= g.t0;
      const bool live = tok < cnt;
      // rows of no token see all of their tile; they are not stored
      const int place = g.place + x * per_tile + (live ? tok : max(cnt, 1) - 1);
      float m_used = -INFINITY, l = 0.f;
      float vsum = 0.f, qsum = 0.f;
      if (Q4 && keys) {
        ok = s2_wait(bar(Q_FULL), n_seg & 1, abort_flag, status, 4);
        ok = __all_sync(0xffffffffu, ok);  // a warp gives up together: what follows needs all of its lanes
        ++n_seg;
        if (ok && has && live) {
          for (int i = 0; i < 8 * kChunks; ++i) {
            const uint32_t at = sQ(x) + (i / 8) * kChunkBytes + r * 128 + (((i % 8) ^ (r & 7)) << 4);
            uint32_t w[4];
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(at));
#pragma unroll
            for (int z = 0; z < 4; ++z)
              qsum += __uint_as_float(w[z] << 16) + __uint_as_float(w[z] & 0xffff0000u);
          }
          qsum *= kQ4Bias;
        }
        mbar_arrive(bar(Q_EMPTY));
      }
      for (int t = g.t0; t < g.t1 && ok; ++t) {
        const int sc = n_sc % kScaleSlots;
        if (t > last) {
          if constexpr (Q4) {
            // the other tile's keys: only counted
            ok = s2_wait(bar(SC_FULL + sc), (n_sc / kScaleSlots) & 1, abort_flag, status, 4);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) mbar_arrive(bar(SC_EMPTY + sc));
            ++n_sc;
            continue;
          } else {
            break;
          }
        }
        ok = s2_wait(bar(S_FULL + x), nS & 1, abort_flag, status, 4);
        if constexpr (Q4) {
          if (ok) ok = s2_wait(bar(SC_FULL + sc), (n_sc / kScaleSlots) & 1, abort_flag, status, 4);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        ++nS;
        const int cmax = min(kT, max(0, place + 1 - t * kT));
        const bool cut = !__all_sync(0xffffffffu, cmax == kT);
        float factor = 1.f;  // by which the maximum's growth shrinks what was summed before
        bool need = false;
        uint32_t s[Q4 ? 64 : kT];   // scores
        const float2 c2 = make_float2(in.scale_log2, in.scale_log2);
        if constexpr (Q4) {
          // Half a tile at a time: 64 scores, their keys' pairs, 32 words of weights.
          const uint32_t scales = sb + L::kScale + sc * 2 * kT * 8;
          const float2 q2 = make_float2(qsum, qsum);
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            Pairs8 pr[2];
            load_pairs(pr[0], scales + half * 64 * 8);
            tmem_ld64(tS + 64 * half, *reinterpret_cast<uint32_t(*)[64]>(&s[0]));
            tmem_wait_ld();
#pragma unroll
            for (int col = 0; col < 64; col += 8) {
              if (col + 8 < 64) load_pairs(pr[(col / 8 + 1) & 1], scales + (half * 64 + col + 8) * 8);
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const float4 a = pr[(col / 8) & 1].p[z];  // {scale, scale, min, min} of two keys
                const int i = col + 2 * z;
                const float2 v = __ffma2_rn(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])),
                                            make_float2(a.x, a.y), __fmul2_rn(make_float2(a.z, a.w), q2));
                s[i] = __float_as_uint(v.x);
                s[i + 1] = __float_as_uint(v.y);
              }
            }
            if (cut) {
#pragma unroll
              for (int col = 0; col < 64; ++col)
                if (64 * half + col >= cmax) s[col] = 0xff800000u;  // -inf
            }
            float mq[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int col = 0; col < 64; col += 4) {
              mq[0] = fmax3(mq[0], __uint_as_float(s[col]), __uint_as_float(s[col + 1]));
              mq[1] = fmax3(mq[1], __uint_as_float(s[col + 2]), __uint_as_float(s[col + 3]));
            }
            const float m_new = fmaxf(m_used, fmaxf(mq[0], mq[1]) * in.scale_log2);
            const bool grow = m_new > m_used + 8.0f;
            float f = 1.f;
            if (grow) {
              // In the second half by a whole number: the factor is a power of two (but for m_to's own rounding, too
              // little to matter), so the first half's weights below, which are bf16 already, stay as exact as they are.
              // Elsewhere to the maximum itself, whose key's weight is then 1 and not rounded (error of ragged 4-bit
              // chunks 0.0022; 0.0024 with whole numbers everywhere).
              float m_to = m_new;
              if (half == 1 && m_used != -INFINITY) m_to = m_used + ceilf(m_new - m_used);
              f = ex2(m_used - m_to);
              l *= f;
              vsum *= f;
              factor *= f;
              need = true;
              m_used = m_to;
            }
            const bool any_grow = __any_sync(0xffffffffu, grow);
            if (half == 1 && any_grow) {  // the first half's weights have been written already
              uint32_t w[32];
              tmem_wait_st();
              tmem_ld32(tS, w);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i)
                w[i] = pack_bf16(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
              tmem_st32(tS, w);
            }
            const float m_exp = base_of(m_used);
            const float2 nm2 = make_float2(-m_exp, -m_exp);
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, vacc = make_float2(0.f, 0.f);
            uint32_t pk[32];
            load_pairs(pr[0], scales + (kT + half * 64) * 8);
#pragma unroll
            for (int col = 0; col < 64; col += 8) {
              if (col + 8 < 64) load_pairs(pr[(col / 8 + 1) & 1], scales + (kT + half * 64 + col + 8) * 8);
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const float4 u = pr[(col / 8) & 1].p[z];
                const int i = col + 2 * z;
                const float2 a =
                    __ffma2_rn(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2, nm2);
                const float2 w = make_float2(ex2(a.x), ex2(a.y));
                acc[z & 1] = __fadd2_rn(acc[z & 1], w);
                vacc = __ffma2_rn(w, make_float2(u.z, u.w), vacc);
                const float2 ws = __fmul2_rn(w, make_float2(u.x, u.y));
                pk[i / 2] = pack_bf16(ws.x, ws.y);
              }
            }
            const float2 sum = __fadd2_rn(acc[0], acc[1]);
            l += sum.x + sum.y;
            vsum += vacc.x + vacc.y;
            tmem_st32(tS + 32 * half, pk);
          }
          mbar_arrive(bar(SC_EMPTY + sc));
          ++n_sc;
        } else {
          tmem_ld128(tS, *reinterpret_cast<uint32_t(*)[kT]>(&s[0]));
          tmem_wait_ld();
          if (cut) {
#pragma unroll
            for (int col = 0; col < kT; ++col)
              if (col >= cmax) s[col] = 0xff800000u;  // -inf
          }
          float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int col = 0; col < kT; col += 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mq[q] = fmax3(mq[q], __uint_as_float(s[col + 2 * q]), __uint_as_float(s[col + 2 * q + 1]));
          }
          const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * in.scale_log2;
          const float m_new = fmaxf(m_used, mx);
          need = m_new > m_used + 8.0f;
          if (need) {
            factor = ex2(m_used - m_new);
            l *= factor;
            m_used = m_new;
          }
          const float m_exp = base_of(m_used);
          const float2 nm2 = make_float2(-m_exp, -m_exp);
          float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int col = 0; col < kT; col += 2) {
            const float2 a =
                __ffma2_rn(make_float2(__uint_as_float(s[col]), __uint_as_float(s[col + 1])), c2, nm2);
            const float2 w = make_float2(ex2(a.x), ex2(a.y));
            acc[(col / 2) & 3] = __fadd2_rn(acc[(col / 2) & 3], w);
            s[col / 2] = pack_bf16(w.x, w.y);
          }
          const float2 sum = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
          l += sum.x + sum.y;
        }
        // (a warp's lanes come together in every tile, since the accesses to tensor memory are all lanes' at once)
        const bool any_need = __any_sync(0xffffffffu, need);
        // S(t) was issued behind O += P V of tile t - 1, so O is complete here
        if (t > g.t0 && any_need) {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            uint32_t o[32];
            tmem_ld32(tO + j * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
            tmem_st32(tO + j * 32, o);
          }
          tmem_wait_st();
        }
        if constexpr (!Q4) tmem_st64(tS, *reinterpret_cast<const uint32_t(*)[64]>(&s[0]));
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(P_FULL + x));
      }
      if (ok && has) {
        ok = s2_wait(bar(O_FULL + x), nO & 1, abort_flag, status, 4);
        ok = __all_sync(0xffffffffu, ok);
        ++nO;
        tc_fence_after();
      }
      // ------------------------------------------------------ rows out
      if (ok) {
        const size_t out = (size_t)(g.tok + x * per_tile + tok) * in.heads + g.h * in.g + r % in.g;
        const float inv = row_scale(l, l, place);
        float4* part = reinterpret_cast<float4*>(in.partial) + partial_at<D>(g.slot, x, 0) + r;
        // four lanes write one row's 64 bytes together: rows of the lanes whose pieces this one writes (or -1)
        int to[4];  // (a call has fewer than 2^31 rows)
#pragma unroll
        for (int z = 0; z < 4; ++z)
          to[z] = __shfl_sync(0xffffffffu, live ? (int)out : -1, (lane & ~3) + z);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          uint32_t o[32];
          if (has) {
            tmem_ld32(tO + j * 32, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          if (g.slot < 0) {
            uint32_t w[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int z = 0; z < 4; ++z)
                w[i][z] = pack_bf16((__uint_as_float(o[8 * i + 2 * z]) + vsum) * inv,
                                    (__uint_as_float(o[8 * i + 2 * z + 1]) + vsum) * inv);
            transpose_pieces(w, lane);
#pragma unroll
            for (int z = 0; z < 4; ++z)
              if (to[z] >= 0)
                *reinterpret_cast<uint4*>(in.o + (size_t)to[z] * D + j * 32 + 8 * (lane & 3)) =
                    make_uint4(w[z][0], w[z][1], w[z][2], w[z][3]);
          } else if (live) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              part[(j * 8 + i) * kT] =
                  make_float4(__uint_as_float(o[4 * i]) + vsum, __uint_as_float(o[4 * i + 1]) + vsum,
                              __uint_as_float(o[4 * i + 2]) + vsum, __uint_as_float(o[4 * i + 3]) + vsum);
          }
          __syncwarp();  // before tensor memory is read again, by all lanes at once
        }
        if (live) {
          if (g.slot < 0) {
            if (in.lse) in.lse[out] = row_lse(m_used, l);
          } else {
            part[(D / 4) * kT] = make_float4(m_used, l, l, 0.f);
          }
        }
        tc_fence_before();  // O has been read: ordered before the next unit's first P_FULL arrival
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

#undef FOR_SEGMENTS
#undef SEGMENT_OF
#undef ISSUE_QK
#undef ISSUE_PV
#undef WAIT_KV
#undef bar
#undef sQ
#undef sKV

// Joins the partial sums of units that the line's cuts run through: blocks
// (i, y) stand for cut i + 1, and share the unit's rows with the blocks of its
// other cuts.  What there is to join they read from the pieces' notes: finding
// it again took each of the many blocks longer than the joining.
// An item is 8 channels of 32 rows, a lane's one of them; with up to 8 pieces a warp takes an item, with more a CTA
// does, its warps sharing the pieces.
// (Six CTAs to a cut, three on an SM, with four pieces' loads in flight: 60 tokens over 8000 keys 33 us; eight, one on an
// SM, eight pieces: 41.)
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 3) s2_cache_chunk_join_kernel(const __grid_constant__ AttnIn in) {
  using namespace chunk;
  constexpr int kW = kJoinThreads / 32, kCols = D / 8, kBatch = 4;
  __shared__ float4 sh_ml[kW][32], sh_o[kW][2][32];
  const int per_tile = kT / in.g;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // every CTA waits, also one with nothing to do: the stream's next launch counts on this one's end alone
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const JoinCut u = static_cast<const JoinCut*>(in.cuts)[blockIdx.x];
  if (u.rows == 0) return;
  const int nth = u.nth * gridDim.y + blockIdx.y, helpers = u.helpers * gridDim.y;
  const bool narrow = u.p1 - u.p0 < kJoinBatch;
  for (int item = narrow ? nth * kW + warp : nth; item < 2 * (kT / 32) * kCols; item += narrow ? helpers * kW : helpers) {
    const int rows = item / kCols, c4 = 2 * (item % kCols);
    const int x = rows / (kT / 32), r0 = rows % (kT / 32) * 32, r = r0 + lane;
    // row of the unit that row r of tile x is; they ascend, so where the first is none all are none
    auto row_at = [&](int y) { return y < per_tile * in.g ? x * per_tile * in.g + y : INT_MAX; };
    if (row_at(r0) >= u.rows) continue;
    const int i = row_at(r);
    const bool live = i < u.rows;
    float m = -INFINITY, l = 0.f, div = 0.f;
    float o[8];
#pragma unroll
    for (int z = 0; z < 8; ++z) o[z] = 0.f;
    const int by = narrow ? 1 : kW;
    for (int p = narrow ? u.p0 : u.p0 + warp; p <= u.p1; p += kBatch * by) {
      float4 ml[kBatch], v[kBatch][2];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        ml[k] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
        v[k][0] = v[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int q = p + k * by;
        if (live && q <= u.p1) {
          const float4* from =
              reinterpret_cast<const float4*>(in.partial) + partial_at<D>(2 * q + (q == u.begin), x, 0) + r;
          ml[k] = from[(D / 4) * kT];
          v[k][0] = from[c4 * kT];
          v[k][1] = from[(c4 + 1) * kT];
        }
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k].x);
      const float base = base_of(top), f = ex2(m - base);
      l *= f;
      div *= f;
#pragma unroll
      for (int z = 0; z < 8; ++z) o[z] *= f;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float e = ex2(ml[k].x - base);
        // a piece in which the row sees no key adds nothing, even where its weights of 0 met values that are not finite
        if (ml[k].y == 0.f) v[k][0] = v[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        l = fmaf(ml[k].y, e, l);
        div = fmaf(ml[k].z, e, div);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          o[4 * h] = fmaf(v[k][h].x, e, o[4 * h]), o[4 * h + 1] = fmaf(v[k][h].y, e, o[4 * h + 1]);
          o[4 * h + 2] = fmaf(v[k][h].z, e, o[4 * h + 2]), o[4 * h + 3] = fmaf(v[k][h].w, e, o[4 * h + 3]);
        }
      }
      m = top;
    }
    if (!narrow) {
      __syncthreads();
      sh_ml[warp][lane] = make_float4(m, l, div, 0.f);
#pragma unroll
      for (int h = 0; h < 2; ++h) sh_o[warp][h][lane] = make_float4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
      __syncthreads();
      if (warp != 0) continue;
#pragma unroll
      for (int w = 1; w < kW; ++w) m = fmaxf(m, sh_ml[w][lane].x);
      l = div = 0.f;
#pragma unroll
      for (int z = 0; z < 8; ++z) o[z] = 0.f;
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const float4 t = sh_ml[w][lane];
        const float e = ex2(t.x - base_of(m));
        l = fmaf(t.y, e, l);
        div = fmaf(t.z, e, div);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 y = sh_o[w][h][lane];
          o[4 * h] = fmaf(y.x, e, o[4 * h]), o[4 * h + 1] = fmaf(y.y, e, o[4 * h + 1]);
          o[4 * h + 2] = fmaf(y.z, e, o[4 * h + 2]), o[4 * h + 3] = fmaf(y.w, e, o[4 * h + 3]);
        }
      }
    }
    if (!live) continue;
    const float inv = row_scale(l, div, u.place + i / in.g);
    const size_t out = (size_t)(u.tok + i / in.g) * in.heads + u.head + i % in.g;
    *reinterpret_cast<uint4*>(in.o + out * D + 4 * c4) =
        make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                   pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
    if (in.lse && c4 == 0) in.lse[out] = row_lse(m, l);
  }
}

template <int D, bool Q4>
static int chunk_impl(const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv, const CacheArgs& c,
                      const AttnIn& in, cudaStream_t stream) {
  using L = chunk::Layout<D, Q4>;
  static_assert(L::kAlloc <= 232448, "shared memory budget");
  cudaError_t e =
      cudaFuncSetAttribute(s2_cache_chunk_kernel<D, Q4>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return (int)e;
  s2_cache_chunk_kernel<D, Q4><<<in.pieces, chunk::threads<Q4>(), L::kAlloc, stream>>>(*tq, *tk, *tv, c, in);
  e = cudaGetLastError();
  if (e != cudaSuccess) return (int)e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(in.pieces - 1, 6);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, s2_cache_chunk_join_kernel<D>, in);
}

int launch_cache_chunk(const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv, const CacheArgs& c,
                       const AttnIn& in, int D, bool q4, cudaStream_t stream) {
  if (D == 64)
    return q4 ? chunk_impl<64, true>(tq, tk, tv, c, in, stream) : chunk_impl<64, false>(tq, tk, tv, c, in, stream);
  return q4 ? chunk_impl<128, true>(tq, tk, tv, c, in, stream) : chunk_impl<128, false>(tq, tk, tv, c, in, stream);
}

static_assert(kChunkPieces * sizeof(JoinCut) <= kCutBytes, "room for the notes");

size_t cache_chunk_partial_bytes(int D) {
  return kCutBytes + (size_t)2 * kChunkPieces * 2 * chunk::kT * (D + 4) * sizeof(float);
}

}  // namespace s2
