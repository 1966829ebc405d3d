// s2attn_cache.cu -- the C ABI of the paged cache (include/s2attn.h): argument
// checks, all before anything is enqueued, and launches.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/s2attn.h"
#include "s2_cache.cuh"
#include "s2_cache_join.cuh"
#include "s2_kernels.h"

namespace {

using s2::report_error;

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Checks of the descriptors that every call shares; fills the kernels' view of them.
int take(const s2_cache* cache, const s2_cache_batch* batch, s2::CacheArgs* a) {
  if (!cache || !batch) return report_error(S2_ERR_INVALID_ARG, "null cache or batch descriptor");
  if (cache->format != S2_CACHE_BF16 && cache->format != S2_CACHE_Q4)
    return report_error(S2_ERR_INVALID_ARG, "unknown cache format %d", cache->format);
  if (cache->pages < 1 || cache->heads < 1 || cache->page_size < 1 || cache->D < 1)
    return report_error(S2_ERR_SHAPE, "pages, heads, page_size and D must be positive");
  if (cache->D != 64 && cache->D != 128)
    return report_error(S2_ERR_UNSUPPORTED, "D=%lld: the cache supports D in {64, 128}", (long long)cache->D);
  const int64_t S = cache->page_size;
  if (S != 16 && S != 32 && S != 64 && S != 128)
    return report_error(S2_ERR_UNSUPPORTED, "page_size=%lld: pages hold 16, 32, 64 or 128 rows", (long long)S);
  if (cache->heads > 65535 || cache->pages >= (int64_t(1) << 31) || cache->pages * cache->heads >= (int64_t(1) << 31))
    return report_error(S2_ERR_UNSUPPORTED, "pages*heads must be below 2^31 and heads below 65536");
  if (cache->pages * cache->heads >= (int64_t(1) << 32) / S)
    return report_error(S2_ERR_UNSUPPORTED, "pages*heads*page_size must be below 2^32");
  if (batch->seqs < 1 || batch->tokens < 1 || batch->table_width < 1)
    return report_error(S2_ERR_SHAPE, "seqs, tokens and table_width must be positive");
  if (batch->max_new < 0 || batch->max_new > batch->tokens)
    return report_error(S2_ERR_SHAPE, "max_new=%lld must be in [0, tokens=%lld]", (long long)batch->max_new,
                        (long long)batch->tokens);
  if (batch->max_len < 0 || batch->table_width >= (int64_t(1) << 30) / S ||
      batch->max_len > batch->table_width * S)
    return report_error(S2_ERR_SHAPE, "max_len=%lld must be in [0, table_width*page_size], which is below 2^30",
                        (long long)batch->max_len);
  if (batch->seqs >= (int64_t(1) << 30) || batch->tokens >= (int64_t(1) << 30))
    return report_error(S2_ERR_UNSUPPORTED, "seqs and tokens must be below 2^30");
  if (!batch->q_starts && batch->tokens != batch->seqs)
    return report_error(S2_ERR_SHAPE, "without q_starts each sequence has one new token (tokens=%lld, seqs=%lld)",
                        (long long)batch->tokens, (long long)batch->seqs);
  const bool q4 = cache->format == S2_CACHE_Q4;
  if (!cache->k || !cache->v || (q4 && (!cache->k_scale || !cache->v_scale)) || !batch->page_table || !batch->seq_lens)
    return report_error(S2_ERR_INVALID_ARG, "null pointer argument");
  if (!q4 && (cache->k_scale || cache->v_scale))
    return report_error(S2_ERR_INVALID_ARG, "a bf16 cache has no scales");
  if (!aligned(cache->k, 16) || !aligned(cache->v, 16) || !aligned(cache->k_scale, 16) || !aligned(cache->v_scale, 16))
    return report_error(S2_ERR_INVALID_ARG, "the cache's pointers must be 16-byte aligned");
  if (!aligned(batch->page_table, 4) || !aligned(batch->seq_lens, 4) || !aligned(batch->q_starts, 4))
    return report_error(S2_ERR_INVALID_ARG, "page_table, seq_lens and q_starts must be 4-byte aligned");
  a->k = cache->k;
  a->v = cache->v;
  a->k_scale = cache->k_scale;
  a->v_scale = cache->v_scale;
  a->table = batch->page_table;
  a->lens = batch->seq_lens;
  a->starts = batch->q_starts;
  a->pages = cache->pages;
  a->heads = (int)cache->heads;
  a->log2s = S == 16 ? 4 : S == 32 ? 5 : S == 64 ? 6 : 7;
  a->B = (int)batch->seqs;
  a->T = (int)batch->tokens;
  a->width = (int)batch->table_width;
  a->status = nullptr;
  return S2_OK;
}

// Rows of a token that are `ld` elements apart hold heads*D elements and stay 16-byte aligned.
int check_rows(const char* name, const void* p, int64_t ld, int64_t elements) {
  if (!p) return report_error(S2_ERR_INVALID_ARG, "null pointer argument (%s)", name);
  if (!aligned(p, 16)) return report_error(S2_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (ld < elements || ld % 8 || ld >= (int64_t(1) << 31))
    return report_error(S2_ERR_SHAPE, "the row stride of %s (%lld) must be a multiple of 8 in [%lld, 2^31)", name,
                        (long long)ld, (long long)elements);
  return S2_OK;
}

// Query heads: a multiple of the key/value heads, at most 128 to one of them.
int check_heads(const s2_cache* cache, int64_t heads) {
  if (heads < 1 || heads % cache->heads)
    return report_error(S2_ERR_SHAPE, "heads=%lld must be a positive multiple of the cache's %lld", (long long)heads,
                        (long long)cache->heads);
  if (heads / cache->heads > 128)
    return report_error(S2_ERR_UNSUPPORTED, "%lld query heads to a key/value head: at most 128",
                        (long long)(heads / cache->heads));
  return S2_OK;
}

// Query rows that share a key/value head in one sequence, as far as the host knows.
int64_t shared_rows(const s2_cache* cache, const s2_cache_batch* batch, int64_t heads) {
  const int64_t n = batch->max_new ? batch->max_new : (batch->tokens + batch->seqs - 1) / batch->seqs;
  return n * (heads / cache->heads);
}

// Which kernel: s2_cache_attn.cu reads (and unpacks) a key once for every 16 query rows and starts quickly,
// s2_cache_chunk.cu once for every 128 and takes 14 us longer to start and end, 17 from 4 bits.  Keys that both go over,
// with what a block of rows costs beside them, decide: the measured times are 8 + 6.5e-5 and 22 + 7e-5 us for each of
// them in bf16, 9 + 4.5e-5 and 26 + 1e-4 in 4 bits, about half of that for half the channels.  us of one and the
// other (tokens over keys, key/value heads; 4 query heads to each, bf16 / 4 bits): 60 over 8000, 8 heads 61 / 49 and 34 /
// 39; 512 over 512 52 / 47 and 28 / 32; 256 over 256 20 / 19 and 27 / 30; 60 over 2000 25 / 23 and 28 / 32; 16 sequences of
// 5 over 2000 42 / 35 and 45 / 57.
bool few_rows(const s2_cache* cache, const s2_cache_batch* batch, int64_t heads) {
  const bool q4 = cache->format == S2_CACHE_Q4;
  const double rows = (double)shared_rows(cache, batch, heads), units = (double)batch->seqs * (double)cache->heads;
  const double len = (double)(batch->max_len ? batch->max_len : batch->table_width * cache->page_size);
  const double few = units * std::ceil(rows / 16) * (len + (q4 ? 256 : 128));
  const double many = units * std::ceil(rows / 128) * (len + 256);
  return (few - (q4 ? 2.2 : 1.0) * many) * ((double)cache->D / 128) <= (q4 ? 4e5 : 2.5e5);
}

int launched(int rc, const char* what) {
  if (rc == 0) return S2_OK;
  return report_error(S2_ERR_CUDA, "%s launch failed: %s", what, cudaGetErrorString((cudaError_t)rc));
}

}  // namespace

extern "C" {

int s2attn_cache_append(const s2_cache* cache, const s2_cache_batch* batch, const void* q, int64_t ldq, const void* k,
                        int64_t ldk, const void* v, int64_t ldv, void* q_out, int64_t heads, const int32_t* positions,
                        double base, double scale, void* stream) {
  s2::CacheArgs a;
  int rc = take(cache, batch, &a);
  if (rc) return rc;
  const int64_t D = cache->D, kv = cache->heads * D;
  if ((rc = check_rows("k", k, ldk, kv)) || (rc = check_rows("v", v, ldv, kv))) return rc;
  const bool rotate = base != 0.0;
  if (rotate && (!(base > 1.0) || !std::isfinite(base) || !(scale > 0.0) || !std::isfinite(scale)))
    return report_error(S2_ERR_INVALID_ARG, "base must be 0 (no rotation) or finite and > 1, scale finite and > 0");
  if (!q != !q_out) return report_error(S2_ERR_INVALID_ARG, "q and q_out go together");
  if (q) {
    if (!rotate) return report_error(S2_ERR_INVALID_ARG, "without a rotation (base 0) there is nothing to do with q");
    if ((rc = check_heads(cache, heads)) || (rc = check_rows("q", q, ldq, heads * D)) ||
        (rc = check_rows("q_out", q_out, heads * D, heads * D)))
      return rc;
  }
  if (!aligned(positions, 4)) return report_error(S2_ERR_INVALID_ARG, "positions must be 4-byte aligned");
  if ((rc = s2::device_status(&a.status))) return rc;
  s2::AppendIn in;
  in.q = static_cast<const __nv_bfloat16*>(q);
  in.k = static_cast<const __nv_bfloat16*>(k);
  in.v = static_cast<const __nv_bfloat16*>(v);
  in.q_out = static_cast<__nv_bfloat16*>(q_out);
  in.positions = positions;
  in.ldq = ldq;
  in.ldk = ldk;
  in.ldv = ldv;
  in.q_heads = q ? (int)heads : 0;
  // a program's calls all have one base and scale: the thread's last table serves them
  thread_local struct { double base, scale; int64_t D; double turns[64]; } last = {0.0, 0.0, 0, {}};
  if (rotate && (last.base != base || last.scale != scale || last.D != D)) {
    for (int j = 0; j < (int)D / 2; ++j)
      last.turns[j] = scale * std::pow(base, -2.0 * j / (double)D) / 6.283185307179586477;
    last.base = base;
    last.scale = scale;
    last.D = D;
  }
  for (int j = 0; j < 64; ++j) in.turns[j] = last.turns[j];
  return launched(s2::launch_cache_append(a, in, (int)D, cache->format == S2_CACHE_Q4, rotate,
                                          static_cast<cudaStream_t>(stream)),
                  "cache append");
}

int s2attn_cache_read(const s2_cache* cache, const s2_cache_batch* batch, void* k_out, void* v_out, void* stream) {
  s2::CacheArgs a;
  int rc = take(cache, batch, &a);
  if (rc) return rc;
  const int64_t kv = cache->heads * cache->D;
  if ((rc = check_rows("k_out", k_out, kv, kv)) || (rc = check_rows("v_out", v_out, kv, kv))) return rc;
  if ((rc = s2::device_status(&a.status))) return rc;
  return launched(s2::launch_cache_read(a, (int)cache->D, cache->format == S2_CACHE_Q4, k_out, v_out,
                                        static_cast<cudaStream_t>(stream)),
                  "cache read");
}

size_t s2attn_cache_attn_workspace_size(const s2_cache* cache, const s2_cache_batch* batch, int64_t heads) {
  s2::CacheArgs a;
  if (take(cache, batch, &a) != S2_OK || check_heads(cache, heads) != S2_OK) return 0;
  // of the kernel that needs more, whichever this batch takes: a program keeps its workspace while sequences come, grow
  // and go, and with them the choice of the kernel changes
  const size_t few = s2::cache_decode_partial_bytes((int)cache->D), many = s2::cache_chunk_partial_bytes((int)cache->D);
  return few > many ? few : many;
}

int s2attn_cache_attn(const s2_cache* cache, const s2_cache_batch* batch, const void* q, int64_t ldq, void* o,
                      float* lse, int64_t heads, void* workspace, size_t workspace_bytes, void* stream) {
  s2::CacheArgs a;
  int rc = take(cache, batch, &a);
  if (rc) return rc;
  if ((rc = check_heads(cache, heads))) return rc;
  const int64_t D = cache->D;
  if ((rc = check_rows("q", q, ldq, heads * D)) || (rc = check_rows("o", o, heads * D, heads * D))) return rc;
  if (heads * batch->tokens >= (int64_t(1) << 31))
    return report_error(S2_ERR_UNSUPPORTED, "tokens*heads must be below 2^31");
  if (!aligned(lse, 4)) return report_error(S2_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  if (!workspace || !aligned(workspace, 256))
    return report_error(S2_ERR_INVALID_ARG, "workspace must be given and 256-byte aligned");
  const size_t need = s2attn_cache_attn_workspace_size(cache, batch, heads);
  if (workspace_bytes < need)
    return report_error(S2_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes,
                        need);
  if ((rc = s2::device_status(&a.status))) return rc;
  s2::AttnIn in;
  in.q = static_cast<const __nv_bfloat16*>(q);
  in.o = static_cast<__nv_bfloat16*>(o);
  in.lse = lse;
  in.partial = static_cast<float*>(workspace);
  in.cuts = nullptr;
  in.ldq = ldq;
  in.heads = (int)heads;
  in.g = (int)(heads / cache->heads);
  const bool q4 = cache->format == S2_CACHE_Q4;
  in.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)D)) * (q4 ? s2::kQ4ScoreUnit : 1.f);
  if (few_rows(cache, batch, heads))
    return launched(s2::launch_cache_decode(a, in, (int)D, q4, shared_rows(cache, batch, heads), batch->max_len,
                                            static_cast<cudaStream_t>(stream)),
                    "cache attention");
  in.cuts = workspace;
  in.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + s2::kCutBytes);
  in.pieces = s2::kChunkPieces;
  in.min_piece = 384;  // keys, 256 of which stand for starting a unit: less is not worth a second launch's reading of partial sums
  const uint64_t S = (uint64_t)cache->page_size, d = (uint64_t)D, blocks = (uint64_t)(cache->pages * cache->heads);
  CUtensorMap tq, tk, tv;
  if ((rc = s2::encode_map(&tq, q, {d, (uint64_t)heads, (uint64_t)batch->tokens}, {d * 2, (uint64_t)ldq * 2},
                           (uint32_t)in.g, (uint32_t)(128 / in.g))))
    return rc;
  if (q4) {
    tk = tv = tq;  // 4-bit pages are not read through tensor maps
  } else if ((rc = s2::encode_map(&tk, cache->k, {d, S, blocks}, {d * 2, S * d * 2}, (uint32_t)S, 1)) ||
             (rc = s2::encode_map(&tv, cache->v, {d, S, blocks}, {d * 2, S * d * 2}, (uint32_t)S, 1))) {
    return rc;
  }
  return launched(s2::launch_cache_chunk(&tq, &tk, &tv, a, in, (int)D, q4, static_cast<cudaStream_t>(stream)),
                  "cache attention");
}

}  // extern "C"
