// C ABI of the serving operators: argument checks, the choice of a form and of
// the split of long caches.
#include <cmath>
#include <cstring>

#include "serve_internal.cuh"

using namespace moe;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

moe_status_t check_cache(const moe_kv_cache* c, KvCacheView* view) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_DTYPE_FP8_E4M3 && c->dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->page_size <= 0 || c->heads <= 0 || c->head_dim <= 0)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return MOE_ERR_INVALID_ARG;
  const bool fp8 = c->dtype == MOE_DTYPE_FP8_E4M3;
  if (fp8 && (c->k_scales == nullptr || c->v_scales == nullptr || !aligned4(c->k_scales) ||
              !aligned4(c->v_scales)))
    return MOE_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return MOE_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0)
    return MOE_ERR_UNSUPPORTED;
  // rows of the cache are counted in 32 bits
  const long long per_page = static_cast<long long>(c->heads) * c->page_size;
  if (per_page > 0x7fffffffll || per_page * c->num_pages > 0x7fffffffll) return MOE_ERR_UNSUPPORTED;
  view->k = static_cast<uint8_t*>(c->k);
  view->v = static_cast<uint8_t*>(c->v);
  view->k_scales = c->k_scales;
  view->v_scales = c->v_scales;
  view->num_pages = c->num_pages;
  view->heads = c->heads;
  view->page_log2 = log2_of(c->page_size);
  return MOE_OK;
}

bool ws_ok(const void* ws) {
  return ws != nullptr && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

bool stride8(int64_t s) { return s % 8 == 0; }

static_assert(MOE_ATTENTION_CTRL_BYTES - MOE_CTRL_BYTES >= 4 * kMaxParts, "a counter per CTA");

}  // namespace

extern "C" {

moe_status_t moe_kv_write(const moe_kv_cache* cache, const void* k, const void* v, int T,
                          int64_t k_stride_t, int64_t k_stride_h, int64_t v_stride_t,
                          int64_t v_stride_h, const int32_t* slots, void* ws, void* stream) {
  KvCacheView c;
  const moe_status_t s = check_cache(cache, &c);
  if (s != MOE_OK) return s;
  if (T < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (k == nullptr || v == nullptr || slots == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned4(slots)) return MOE_ERR_INVALID_ARG;
  if (!stride8(k_stride_t) || !stride8(k_stride_h) || !stride8(v_stride_t) ||
      !stride8(v_stride_h))
    return MOE_ERR_INVALID_ARG;
  if (static_cast<long long>(T) * c.heads > 0x7fffffffll) return MOE_ERR_UNSUPPORTED;
  if (!ws_ok(ws)) return MOE_ERR_WORKSPACE;
  return cuda_status(launch_kv_write(c, cache->head_dim, cache->dtype == MOE_DTYPE_FP8_E4M3, k, v,
                                     T, k_stride_t, k_stride_h, v_stride_t, v_stride_h, slots,
                                     static_cast<Ctrl*>(ws), static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_kv_read(const moe_kv_cache* cache, const int32_t* block_table, int table_stride,
                         const int32_t* cu_rows, const int32_t* starts, int B, int rows,
                         void* k_out, void* v_out, void* ws, void* stream) {
  KvCacheView c;
  const moe_status_t s = check_cache(cache, &c);
  if (s != MOE_OK) return s;
  if (B < 0 || rows < 0 || table_stride < 0) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (B == 0 || (block_table == nullptr && table_stride > 0) || cu_rows == nullptr ||
      k_out == nullptr || v_out == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(k_out) || !aligned16(v_out)) return MOE_ERR_INVALID_ARG;
  if (c.heads > 0x7fffffff / (16 * 16)) return MOE_ERR_UNSUPPORTED;
  if (!ws_ok(ws)) return MOE_ERR_WORKSPACE;
  return cuda_status(launch_kv_read(c, cache->head_dim, cache->dtype == MOE_DTYPE_FP8_E4M3,
                                    block_table, table_stride, cu_rows, starts, B, rows, k_out,
                                    v_out, static_cast<Ctrl*>(ws),
                                    static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_paged_attention(const moe_attention_args* a, void* ws, size_t ws_bytes,
                                 void* stream) {
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  AttnParams p;
  std::memset(&p, 0, sizeof(p));
  const moe_status_t s = check_cache(&a->cache, &p.c);
  if (s != MOE_OK) return s;
  if (a->B < 0 || a->T < 0 || a->q_heads <= 0 || a->max_q < 0 || a->max_kv < 0 ||
      a->table_stride < 0 || a->window < 0)
    return MOE_ERR_INVALID_ARG;
  if (a->q_heads % p.c.heads != 0) return MOE_ERR_INVALID_ARG;
  if (a->causal != 0 && a->causal != 1) return MOE_ERR_INVALID_ARG;
  if (a->window > 0 && a->causal == 0) return MOE_ERR_INVALID_ARG;
  if (!(a->softcap >= 0.0f) || !std::isfinite(a->softcap) || !std::isfinite(a->scale))
    return MOE_ERR_INVALID_ARG;
  if (a->T == 0 || a->B == 0 || a->max_q == 0) return MOE_OK;
  if (a->q == nullptr || a->out == nullptr || a->cu_q == nullptr || a->kv_lens == nullptr ||
      (a->block_table == nullptr && a->table_stride > 0))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(a->q) || !aligned16(a->out) || !aligned4(a->lse)) return MOE_ERR_INVALID_ARG;
  if (!stride8(a->q_stride_t) || !stride8(a->q_stride_h) || !stride8(a->out_stride_t) ||
      !stride8(a->out_stride_h))
    return MOE_ERR_INVALID_ARG;
  const int group = a->q_heads / p.c.heads;
  const long long room = static_cast<long long>(a->table_stride) * a->cache.page_size;
  const long long rows = static_cast<long long>(a->max_q) * group;
  if (room > 0x7fffffffll - 512 || rows > 0x7fffffffll - 512) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->T) * a->q_heads > 0x7fffffffll) return MOE_ERR_UNSUPPORTED;
  if (!ws_ok(ws) || ws_bytes < MOE_ATTENTION_CTRL_BYTES) return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;

  const bool fp8 = a->cache.dtype == MOE_DTYPE_FP8_E4M3;
  const int D = a->cache.head_dim;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.q_st = a->q_stride_t;
  p.q_sh = a->q_stride_h;
  p.o_st = a->out_stride_t;
  p.o_sh = a->out_stride_h;
  p.cu_q = a->cu_q;
  p.kv_lens = a->kv_lens;
  p.table = a->block_table;
  p.table_stride = a->table_stride;
  p.B = a->B;
  p.T = a->T;
  p.q_heads = a->q_heads;
  p.group = group;
  p.max_q = a->max_q;
  p.scale = a->scale == 0.0f ? 1.0f / std::sqrt(static_cast<float>(D)) : a->scale;
  p.softcap = a->softcap;
  p.window = a->window;
  p.causal = a->causal;
  p.ctrl = static_cast<Ctrl*>(ws);
  p.counters = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(ws) + MOE_CTRL_BYTES);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + MOE_ATTENTION_CTRL_BYTES);
  p.timeout_ns = wait_limit_ns();
  p.drop_producer = loads_dropped() ? 1 : 0;

  // Few rows per cache head: one tile of them, keys as the tensor core's rows, bound by HBM.
  // More: 256-row tiles.  (8192 keys x 4 heads x D 128, us in the first form / in the second.
  // BF16, 64 rows: 38 sequences 109 / 109, 6 sequences 34 / 38.  FP8, whose small weights the
  // first form checks: 48 rows 79 / 139 and 29 / 42; 64 rows, where its registers spill, 169 / 140
  // and 46 / 46.  Scores four times as large, whose weights ask for a second pass in most tiles:
  // 48 rows FP8 204 / 144 and 48 / 44.)
  const bool few = rows <= (fp8 ? 48 : 64);
  const int tile_rows = !few ? kTileRows : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 48 ? 48 : 64;
  p.row_tiles = static_cast<int>((rows + tile_rows - 1) / tile_rows);
  const long long tiles = static_cast<long long>(a->B) * p.c.heads * p.row_tiles;
  if (tiles > 0x7fffffffll / 2) return MOE_ERR_UNSUPPORTED;
  p.part_rows = rows < tile_rows ? static_cast<int>((rows + 15) / 16 * 16) : tile_rows;
  const long long part_bytes = static_cast<long long>(p.part_rows) * (D + 2) * 4;
  const long long room_parts =
      static_cast<long long>((ws_bytes - MOE_ATTENTION_CTRL_BYTES) / part_bytes);
  // The keys a tile may see, by the caller's hint
  long long span = a->max_kv > 0 && a->max_kv < room ? a->max_kv : room;
  const long long reach = static_cast<long long>(a->window) + tile_rows / group + 128;
  if (a->window > 0 && reach < span) span = reach;
  const long long most = (span + 255) / 256;      // parts of at least 256 keys
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (few) {
    // Fewer tiles than places for CTAs on the SMs: a CTA for every place, which share the
    // tiles' keys among them (in parts of at least 256; the kernel goes by kv_lens).
    const long long places =
        static_cast<long long>(attention_rows_places(tile_rows, D, fp8)) * sms;
    const bool share = tiles < places && most > 1 && places <= room_parts && places <= kMaxParts;
    p.splits = share ? static_cast<int>(places) : 1;
    p.whole = static_cast<int>(share ? places : tiles);
    p.span = static_cast<int>(a->window > 0 && reach < room ? reach : room);
    return cuda_status(launch_attention_rows(p, tile_rows, D, fp8, st));
  }
  // One tile per SM at a time.  The tiles past the last full round, which are the early rows,
  // are cut into the number of parts that takes the least time by this estimate: about 1.5 us
  // for 128 keys, and 20 us more for a part (its 133 KB written and read again; 2 x 16
  // heads of 8192 rows and keys: 565 us whole, 623 us with the last 112 tiles in 4 parts;
  // a 4096-row chunk at 16384 keys: 711 us whole, 688 us with its last 56 in 2; all with
  // BF16 and D = 128.  FP8's tiles take longer and D = 64's parts are half as large: not fitted).
  // Early rows see fewer keys by the new tokens after them, but not those of single tokens or
  // drafted runs beside a long chunk (what the longest sequence leaves to each of the others is
  // then at most a row tile): they see all their keys.  (8192 tokens and one token over 8192
  // positions, 8 heads, BF16 / FP8: 509 / 698 us by the chunk's length, 477 / 645 so.  Taking the
  // others' average in ragged prompts and chunks too: 8192 and 5000 tokens 620 / 831 us whole and
  // 658 / 870 in parts, five chunks of 2000 to 4100 595 / 796 and 640 / 841.)
  const long long rest = tiles % sms;
  const bool beside = a->B > 1 && static_cast<long long>(a->T - a->max_q) * group <=
                                      static_cast<long long>(a->B - 1) * tile_rows;
  long long seen = span;
  if (a->causal != 0 && !beside) {
    const long long late = p.row_tiles - 1 - rest / (static_cast<long long>(a->B) * p.c.heads);
    seen -= late * tile_rows / group;
    if (seen < 0) seen = 0;
  }
  const double tile_us = 1.5 * static_cast<double>(seen) / 128.0;
  long long splits = 1;
  double best = tile_us;
  for (long long s = 2; s <= 16 && s <= most && rest * s <= room_parts; ++s) {
    const double us = static_cast<double>((rest * s + sms - 1) / sms) * (tile_us / s + 20.0);
    if (us < best) {
      best = us;
      splits = s;
    }
  }
  p.splits = static_cast<int>(splits);
  p.whole = static_cast<int>(splits > 1 ? tiles - rest : tiles);
  return cuda_status(launch_attention_tiles(p, D, fp8, st));
}

moe_status_t moe_verify_draft(const moe_verify_args* a, void* ws, void* stream) {
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  if (a->dtype != MOE_DTYPE_F32 && a->dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (a->B < 0 || a->n <= 0 || a->V <= 0) return MOE_ERR_INVALID_ARG;
  if (a->B == 0) return MOE_OK;
  if (a->p == nullptr || a->q == nullptr || a->draft == nullptr || a->u_accept == nullptr ||
      a->u_sample == nullptr || a->accepted == nullptr || a->tokens == nullptr)
    return MOE_ERR_INVALID_ARG;
  const uintptr_t esize = a->dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(a->p) % esize != 0 ||
      reinterpret_cast<uintptr_t>(a->q) % esize != 0)
    return MOE_ERR_INVALID_ARG;
  if (a->n > 32 || a->V >= (1 << 24) || a->B > 0x7fffffff / 8) return MOE_ERR_UNSUPPORTED;
  if (!ws_ok(ws)) return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  return cuda_status(
      launch_verify(*a, static_cast<Ctrl*>(ws), sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
