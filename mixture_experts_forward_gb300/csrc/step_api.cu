// C ABI of the operators between the serving operators: the step's plan, rotary positions, the
// few-token experts and the logits.  Argument checks and launches.
#include <cmath>

#include "serve_internal.cuh"

using namespace moe;

namespace {

bool aligned_to(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool stride8(int64_t s) { return s % 8 == 0; }
bool ws_ok(const void* ws) { return ws != nullptr && aligned_to(ws, 256); }

moe_status_t check_pages(const moe_page_state* p) {
  if (p == nullptr) return MOE_ERR_INVALID_ARG;
  if (p->B < 0 || p->table_stride < 0 || p->page_size <= 0 || p->free_capacity < 0)
    return MOE_ERR_INVALID_ARG;
  if ((p->held == nullptr && p->B > 0) || p->free_count == nullptr ||
      (p->block_table == nullptr && p->table_stride > 0 && p->B > 0) ||
      (p->free_pages == nullptr && p->free_capacity > 0))
    return MOE_ERR_INVALID_ARG;
  if (!aligned_to(p->held, 4) || !aligned_to(p->free_count, 4) || !aligned_to(p->block_table, 4) ||
      !aligned_to(p->free_pages, 4))
    return MOE_ERR_INVALID_ARG;
  if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1)) != 0)
    return MOE_ERR_UNSUPPORTED;
  if (p->B > kMaxPlanned) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(p->B) * p->table_stride > 0x7fffffffll ||
      static_cast<long long>(p->table_stride) * p->page_size > 0x7fffffffll - 512)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The arguments of moe_forward that the few-token layer reads.
moe_status_t check_few(const moe_forward_args* f) {
  if (f == nullptr || f->M <= 0 || f->K <= 0 || f->N <= 0 || f->E <= 0 || f->top_k <= 0)
    return MOE_ERR_INVALID_ARG;
  const bool fp8 = f->dtype == MOE_DTYPE_FP8_E4M3;
  if (!fp8 && f->dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (!(f->softcap >= 0.0f) || !std::isfinite(f->softcap)) return MOE_ERR_INVALID_ARG;
  if (f->gated != 0 && f->gated != 1) return MOE_ERR_INVALID_ARG;
  if (fp8 && f->gated == 0) return MOE_ERR_UNSUPPORTED;     // one product: moe_forward
  if (f->M > MOE_FEW_TOKENS || f->E > 1024 || f->top_k > 32 || f->top_k > f->E)
    return MOE_ERR_UNSUPPORTED;
  if (f->K % (fp8 ? 128 : 64) != 0 || f->N % 128 != 0 || f->K > 32768 || f->N > 32768)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t few_bytes(const moe_forward_args* f) {
  return kFewWsBytes + static_cast<size_t>(f->M) * f->top_k * f->N * 4;
}

}  // namespace

extern "C" {

moe_status_t moe_plan_step(const moe_page_state* pages, const int32_t* lens,
                           const int32_t* new_lens, int rows, int num_pages, int32_t* slots,
                           int32_t* positions, int32_t* cu_q, int32_t* kv_lens, void* ws,
                           void* stream) {
  const moe_status_t s = check_pages(pages);
  if (s != MOE_OK) return s;
  if (rows < 0 || num_pages < 0 || cu_q == nullptr) return MOE_ERR_INVALID_ARG;
  if (pages->B > 0 && (lens == nullptr || new_lens == nullptr || kv_lens == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (slots == nullptr || positions == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(lens, 4) || !aligned_to(new_lens, 4) || !aligned_to(slots, 4) ||
      !aligned_to(positions, 4) || !aligned_to(cu_q, 4) || !aligned_to(kv_lens, 4))
    return MOE_ERR_INVALID_ARG;
  if (rows > (1 << 30) || static_cast<long long>(num_pages) * pages->page_size > 0x7fffffffll)
    return MOE_ERR_UNSUPPORTED;
  if (!ws_ok(ws)) return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  return cuda_status(launch_plan_step(*pages, lens, new_lens, rows, num_pages, slots, positions,
                                      cu_q, kv_lens, static_cast<Ctrl*>(ws), sms,
                                      static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_release_pages(const moe_page_state* pages, const int32_t* keep, void* ws,
                               void* stream) {
  const moe_status_t s = check_pages(pages);
  if (s != MOE_OK) return s;
  if (pages->B == 0) return MOE_OK;
  if (keep == nullptr || !aligned_to(keep, 4)) return MOE_ERR_INVALID_ARG;
  if (!ws_ok(ws)) return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  return cuda_status(launch_release_pages(*pages, keep, static_cast<Ctrl*>(ws), sms,
                                          static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_rotary_table(int rotary_dim, double base, moe_rope_scaling_t scaling,
                              double factor, double original, double low, double high,
                              uint64_t* table) {
  if (table == nullptr || rotary_dim <= 0 || rotary_dim % 2 != 0) return MOE_ERR_INVALID_ARG;
  if (rotary_dim > 512) return MOE_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !std::isfinite(base) || !(factor > 0.0) || !std::isfinite(factor))
    return MOE_ERR_INVALID_ARG;
  if (scaling < MOE_ROPE_NONE || scaling > MOE_ROPE_INDEX) return MOE_ERR_INVALID_ARG;
  const bool blended = scaling == MOE_ROPE_TURNS || scaling == MOE_ROPE_INDEX;
  if (blended && (!(original > 0.0) || !std::isfinite(original) || !(low > 0.0) || !(high > low) ||
                  !std::isfinite(high)))
    return MOE_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586;
  double from = 0.0, to = 1.0;
  if (scaling == MOE_ROPE_INDEX) {
    // the index of the pair that makes so many turns over the trained context
    auto index = [&](double turns) {
      return rotary_dim * std::log(original / (turns * two_pi)) / (2.0 * std::log(base));
    };
    from = std::fmax(std::floor(index(high)), 0.0);
    to = std::fmin(std::ceil(index(low)), rotary_dim - 1.0);
    if (!(to > from)) to = from + 0.001;
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double theta = std::pow(base, -2.0 * i / rotary_dim);
    double keep = 1.0;
    if (scaling == MOE_ROPE_LINEAR) keep = 0.0;
    if (scaling == MOE_ROPE_TURNS) keep = (original * theta / two_pi - low) / (high - low);
    if (scaling == MOE_ROPE_INDEX) keep = 1.0 - (i - from) / (to - from);
    keep = std::fmin(1.0, std::fmax(0.0, keep));
    double turns = (theta * keep + theta / factor * (1.0 - keep)) / two_pi;
    if (!std::isfinite(turns)) return MOE_ERR_INVALID_ARG;   // (a factor near the end of the type)
    turns -= std::floor(turns);                      // (a factor below 1 / 2 pi)
    // below 1, so the product is below 2^64 (53 bits of it, the rest zero)
    table[i] = static_cast<uint64_t>(turns * 18446744073709551616.0);
  }
  return MOE_OK;
}

moe_status_t moe_rotary(const moe_rotary_args* a, void* ws, void* stream) {
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  const bool cached = a->cache.k != nullptr;
  KvCacheView view;
  if (cached) {
    const moe_status_t s = check_cache(&a->cache, &view);
    if (s != MOE_OK) return s;
    if (a->kv_heads != a->cache.heads || a->head_dim != a->cache.head_dim)
      return MOE_ERR_INVALID_ARG;
  }
  if (a->T < 0 || a->q_heads < 0 || a->kv_heads < 0 || a->head_dim <= 0 || a->rotary_dim <= 0)
    return MOE_ERR_INVALID_ARG;
  if (a->rotary_dim > a->head_dim) return MOE_ERR_INVALID_ARG;
  if (a->interleaved != 0 && a->interleaved != 1) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(a->amplitude)) return MOE_ERR_INVALID_ARG;
  if (a->head_dim % 16 != 0 || a->head_dim > 256 || a->rotary_dim % 16 != 0)
    return MOE_ERR_UNSUPPORTED;
  if (a->T == 0 || a->q_heads + static_cast<long long>(a->kv_heads) == 0) return MOE_OK;
  if (a->table == nullptr || !aligned_to(a->table, 8) || a->positions == nullptr ||
      !aligned_to(a->positions, 4))
    return MOE_ERR_INVALID_ARG;
  if (a->q_heads > 0 && (a->q == nullptr || a->q_out == nullptr || !aligned16(a->q) ||
                         !aligned16(a->q_out) || !stride8(a->q_stride_t) ||
                         !stride8(a->q_stride_h) || !stride8(a->q_out_stride_t) ||
                         !stride8(a->q_out_stride_h)))
    return MOE_ERR_INVALID_ARG;
  if (a->kv_heads > 0 && (a->k == nullptr || !aligned16(a->k) || !stride8(a->k_stride_t) ||
                          !stride8(a->k_stride_h)))
    return MOE_ERR_INVALID_ARG;
  if (a->kv_heads > 0 && !cached && (a->k_out == nullptr || !aligned16(a->k_out) ||
                                     !stride8(a->k_out_stride_t) || !stride8(a->k_out_stride_h)))
    return MOE_ERR_INVALID_ARG;
  if (cached && (a->v == nullptr || !aligned16(a->v) || !stride8(a->v_stride_t) ||
                 !stride8(a->v_stride_h) || a->slots == nullptr || !aligned_to(a->slots, 4)))
    return MOE_ERR_INVALID_ARG;
  // a CTA's pieces are counted in 32 bits
  if (static_cast<long long>(a->q_heads) + 2ll * a->kv_heads > (1ll << 20)) return MOE_ERR_UNSUPPORTED;
  if (cached && !ws_ok(ws)) return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  return cuda_status(launch_rotary(*a, cached ? &view : nullptr, static_cast<Ctrl*>(ws), sms,
                                   static_cast<cudaStream_t>(stream)));
}

size_t moe_few_workspace_size(const moe_forward_args* args) {
  return check_few(args) == MOE_OK ? (few_bytes(args) + 255) / 256 * 256 : 0;
}

moe_status_t moe_forward_few(const moe_forward_args* args, void* out, void* ws, size_t ws_bytes,
                             void* stream) {
  const moe_status_t s = check_few(args);
  if (s != MOE_OK) return s;
  if (args->logits == nullptr || args->x == nullptr || args->w == nullptr || args->w2 == nullptr ||
      out == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(args->x) || !aligned16(args->w) || !aligned16(args->w2) ||
      !aligned_to(args->logits, 4) || !aligned_to(out, 2))
    return MOE_ERR_INVALID_ARG;
  if (args->dtype == MOE_DTYPE_FP8_E4M3 &&
      (args->w_scales == nullptr || args->w2_scales == nullptr || !aligned_to(args->w_scales, 4) ||
       !aligned_to(args->w2_scales, 4)))
    return MOE_ERR_INVALID_ARG;
  if (!ws_ok(ws) || ws_bytes < few_bytes(args)) return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  return cuda_status(launch_few_experts(*args, out, static_cast<uint8_t*>(ws), sms,
                                        static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_adjust_logits(const moe_logits_args* a, void* ws, void* stream) {
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  if (a->dtype != MOE_DTYPE_F32 && a->dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (a->B < 0 || a->m <= 0 || a->V <= 0 || a->history_stride < 0 || a->biases < 0)
    return MOE_ERR_INVALID_ARG;
  if (a->probabilities != 0 && a->probabilities != 1) return MOE_ERR_INVALID_ARG;
  if (a->m > 33 || a->V > 262144 || a->biases > 1024) return MOE_ERR_UNSUPPORTED;
  if (a->history != nullptr && a->history_stride > (1 << 20) - 64) return MOE_ERR_UNSUPPORTED;
  // a CTA for each eighth of a row, counted in 32 bits
  if (static_cast<long long>(a->B) * a->m > 0x7fffffffll / 64) return MOE_ERR_UNSUPPORTED;
  if (a->B == 0) return MOE_OK;
  if (a->logits == nullptr || a->out == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(a->logits, a->dtype == MOE_DTYPE_F32 ? 4 : 2)) return MOE_ERR_INVALID_ARG;
  if (a->biases > 0 && (a->bias_tokens == nullptr || a->bias_values == nullptr))
    return MOE_ERR_INVALID_ARG;
  const void* words[] = {a->out, a->history, a->history_lens, a->prompt_lens, a->draft,
                         a->repetition, a->presence, a->frequency, a->temperature,
                         a->bias_tokens, a->bias_values, a->mask};
  for (const void* w : words)
    if (!aligned_to(w, 4)) return MOE_ERR_INVALID_ARG;
  if (!ws_ok(ws)) return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  return cuda_status(launch_adjust_logits(*a, static_cast<Ctrl*>(ws), sms,
                                          static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
