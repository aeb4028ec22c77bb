// api_cache.cu -- the C entry points of the cache and sampling operators: host-side checks
// and launches.  Every check runs before any launch; a failed one touches no device memory.
#include <math.h>
#include <stdint.h>

#include "kernels.h"
#include "pspec.h"

namespace {

using namespace pspec;

bool dtype_ok(pspec_dtype d) { return d == PSPEC_F32 || d == PSPEC_BF16; }
long long elem_bytes(pspec_dtype d) { return d == PSPEC_BF16 ? 2 : 4; }
bool aligned(const void* p, long long n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

struct Span {
  const void* p;
  long long bytes;
};

bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// a * b in *out; false where it passes 2^62 (the sizes here are products of host integers)
bool mul(long long a, long long b, long long* out) {
  if (a < 0 || b < 0) return false;
  if (b != 0 && a > (1LL << 62) / b) return false;
  *out = a * b;
  return true;
}

}  // namespace

extern "C" {

pspec_status pspec_append_kv(const pspec_append_args* a, cudaStream_t stream) {
  if (!a) return PSPEC_ERR_INVALID_ARG;
  if (a->T < 0 || a->Hkv < 1 || a->D < 16 || a->D > 512 || a->D % 16 != 0) return PSPEC_ERR_INVALID_ARG;
  if (a->rot < 0 || a->rot > a->D || a->rot % 2 != 0) return PSPEC_ERR_INVALID_ARG;
  if (a->block_size < 1 || a->num_blocks < 1 || !dtype_ok(a->dtype) || !a->err) return PSPEC_ERR_INVALID_ARG;
  if (a->cache != PSPEC_CACHE_ROWS && a->cache != PSPEC_CACHE_E2M1) return PSPEC_ERR_INVALID_ARG;
  if (a->q && (a->Hq < 1 || !a->q_out)) return PSPEC_ERR_INVALID_ARG;
  const long long e = elem_bytes(a->dtype);
  const bool e2m1 = a->cache == PSPEC_CACHE_E2M1;
  long long slots, cache_rows, page_bytes, scale_bytes = 0, kv_row, q_row = 0, kv_bytes, q_bytes = 0;
  if (!mul(a->num_blocks, a->block_size, &slots) || !mul(slots, a->Hkv, &cache_rows) ||
      !mul(cache_rows, e2m1 ? a->D / 2 : a->D * e, &page_bytes) || !mul(a->Hkv, a->D, &kv_row) ||
      !mul(kv_row * e, a->T, &kv_bytes))
    return PSPEC_ERR_INVALID_ARG;
  if (e2m1) scale_bytes = cache_rows * (a->D / 16);
  if (a->q && (!mul(a->Hq, a->D, &q_row) || !mul(q_row * e, a->T, &q_bytes))) return PSPEC_ERR_INVALID_ARG;
  if (kv_row > 0x7fffffffLL || q_row > 0x7fffffffLL) return PSPEC_ERR_INVALID_ARG;
  long long tmp;
  if (a->k_stride < kv_row || a->v_stride < kv_row || (a->q && a->q_stride < q_row) ||
      !mul(a->T, a->k_stride, &tmp) || !mul(a->T, a->v_stride, &tmp) || (a->q && !mul(a->T, a->q_stride, &tmp)))
    return PSPEC_ERR_INVALID_ARG;
  if (a->T == 0) { record_launches(0); return PSPEC_OK; }
  if (!a->k || !a->v || !a->positions || !a->slot_mapping || !a->k_pages || !a->v_pages ||
      (a->rot > 0 && !a->inv_freq))
    return PSPEC_ERR_INVALID_ARG;
  if (e2m1 && (!a->k_block_scales || !a->v_block_scales)) return PSPEC_ERR_INVALID_ARG;
  if (!aligned(a->k, e) || !aligned(a->v, e) || (a->q && (!aligned(a->q, e) || !aligned(a->q_out, e))) ||
      !aligned(a->k_out, e) || !aligned(a->v_out, e) || !aligned(a->k_pages, 16) || !aligned(a->v_pages, 16) ||
      !aligned(a->positions, 4) || !aligned(a->slot_mapping, 8) || !aligned(a->err, 4) ||
      !aligned(a->inv_freq, 4) || !aligned(a->k_scale, 4) || !aligned(a->v_scale, 4))
    return PSPEC_ERR_INVALID_ARG;

  const Span outs[] = {{a->q ? a->q_out : nullptr, q_bytes}, {a->k_out, kv_bytes}, {a->v_out, kv_bytes},
                       {a->k_pages, page_bytes}, {a->v_pages, page_bytes},
                       {e2m1 ? a->k_block_scales : nullptr, scale_bytes},
                       {e2m1 ? a->v_block_scales : nullptr, scale_bytes}};
  const long long T1 = a->T - 1;
  const Span ins[] = {{a->q, (T1 * a->q_stride + q_row) * e}, {a->k, (T1 * a->k_stride + kv_row) * e},
                      {a->v, (T1 * a->v_stride + kv_row) * e}, {a->positions, a->T * 4LL},
                      {a->slot_mapping, a->T * 8LL}, {a->inv_freq, a->rot * 2LL},
                      {e2m1 ? a->k_scale : nullptr, a->Hkv * 4LL}, {e2m1 ? a->v_scale : nullptr, a->Hkv * 4LL}};
  constexpr int n_out = sizeof(outs) / sizeof(outs[0]);
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return PSPEC_ERR_INVALID_ARG;
    for (const Span& s : ins)
      if (overlap(outs[i], s)) return PSPEC_ERR_INVALID_ARG;
  }

  AppendLaunch L{};
  L.a = *a;
  L.slots = slots;
  // eight elements of a head at a time, in 16-byte pieces
  L.vec_q = a->q && aligned(a->q, 16) && a->q_stride * e % 16 == 0;
  L.vec_k = aligned(a->k, 16) && a->k_stride * e % 16 == 0;
  L.vec_v = aligned(a->v, 16) && a->v_stride * e % 16 == 0;
  L.vec_qo = a->q && aligned(a->q_out, 16);
  L.vec_ko = aligned(a->k_out, 16);
  L.vec_vo = aligned(a->v_out, 16);
  if (launch_append(L, stream) != cudaSuccess) return PSPEC_ERR_CUDA;
  record_launches(1);
  return PSPEC_OK;
}

size_t pspec_attend_workspace_bytes(void) { return attend_workspace_bytes(); }

pspec_status pspec_attend(const pspec_attend_args* a, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  if (!a) return PSPEC_ERR_INVALID_ARG;
  if (a->T < 0 || a->B < 0 || a->Hkv < 1 || a->Hq < a->Hkv || a->Hq % a->Hkv != 0 || a->D < 1)
    return PSPEC_ERR_INVALID_ARG;
  if (a->block_size < 1 || a->num_blocks < 1 || a->max_blocks < 1 || !dtype_ok(a->dtype) || !a->err ||
      !isfinite(a->scale))
    return PSPEC_ERR_INVALID_ARG;
  if (a->D != 64 && a->D != 128) return PSPEC_ERR_UNSUPPORTED;
  const long long e = elem_bytes(a->dtype);
  long long q_row, out_bytes, slots, cache_rows, tmp;
  if (!mul(a->Hq, a->D, &q_row) || !mul(q_row * e, a->T, &out_bytes) || !mul(a->num_blocks, a->block_size, &slots) ||
      !mul(slots, (long long)a->Hkv * a->D, &cache_rows) || a->q_stride < q_row || !mul(a->T, a->q_stride, &tmp) ||
      (long long)a->Hkv * a->block_size > 0x7fffffffLL)
    return PSPEC_ERR_INVALID_ARG;
  if (a->T == 0 || a->B == 0) { record_launches(0); return PSPEC_OK; }
  if (!a->q || !a->k_pages || !a->v_pages || !a->k_block_scales || !a->v_block_scales || !a->block_table ||
      !a->qsl || !a->positions || !a->seq_lens || !a->out)
    return PSPEC_ERR_INVALID_ARG;
  if (!aligned(a->q, e) || !aligned(a->out, 16) || !aligned(a->k_pages, 16) || !aligned(a->v_pages, 16) ||
      !aligned(a->k_block_scales, 16) || !aligned(a->v_block_scales, 16) || !aligned(a->k_scale, 4) ||
      !aligned(a->v_scale, 4) || !aligned(a->block_table, 4) || !aligned(a->qsl, 4) ||
      !aligned(a->positions, 4) || !aligned(a->seq_lens, 4) || !aligned(a->lse, 4) || !aligned(a->err, 4))
    return PSPEC_ERR_INVALID_ARG;
  const Span q = {a->q, ((a->T - 1) * a->q_stride + q_row) * e}, o = {a->out, out_bytes},
             l = {a->lse, 4LL * a->T * a->Hq};
  if (overlap(q, o) || overlap(q, l) || overlap(o, l)) return PSPEC_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < attend_workspace_bytes())
    return PSPEC_ERR_WORKSPACE;
  AttendLaunch L{};
  L.a = *a;
  L.cnt = static_cast<int*>(workspace);
  L.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + attend_counter_bytes());
  if (launch_attend(L, stream) != cudaSuccess) return PSPEC_ERR_CUDA;
  record_launches(1);
  return PSPEC_OK;
}

pspec_status pspec_sample_filtered(const pspec_filter_args* a, cudaStream_t stream) {
  if (!a) return PSPEC_ERR_INVALID_ARG;
  if (a->B < 0 || a->K < 1 || a->V < 1 || a->ld < a->V || !dtype_ok(a->dtype) || !a->err)
    return PSPEC_ERR_INVALID_ARG;
  if (a->B == 0) { record_launches(0); return PSPEC_OK; }
  if (!a->logits || !a->uniforms || !a->tokens) return PSPEC_ERR_INVALID_ARG;
  if (!aligned(a->logits, elem_bytes(a->dtype)) || !aligned(a->uniforms, 4) || !aligned(a->temperature, 4) ||
      !aligned(a->top_k, 4) || !aligned(a->top_p, 4) || !aligned(a->min_p, 4) || !aligned(a->tokens, 4) ||
      !aligned(a->probs, 4) || !aligned(a->err, 4))
    return PSPEC_ERR_INVALID_ARG;
  long long tmp;
  if (!mul((long long)a->B * a->K, a->ld, &tmp)) return PSPEC_ERR_INVALID_ARG;
  if ((long long)a->B * a->K * 16 >= 0x7fffffffLL || a->V > PSPEC_FILTER_MAX_V) return PSPEC_ERR_UNSUPPORTED;
  const long long rows = (long long)a->B * a->K, e = elem_bytes(a->dtype);
  const Span outs[] = {{a->tokens, 4 * rows}, {a->probs, 4 * rows}};
  const Span ins[] = {{a->logits, ((rows - 1) * a->ld + a->V) * e}, {a->uniforms, 4 * rows},
                      {a->temperature, 4LL * a->B}, {a->top_k, 4LL * a->B}, {a->top_p, 4LL * a->B},
                      {a->min_p, 4LL * a->B}};
  if (overlap(outs[0], outs[1])) return PSPEC_ERR_INVALID_ARG;
  for (const Span& o : outs)
    for (const Span& s : ins)
      if (overlap(o, s)) return PSPEC_ERR_INVALID_ARG;
  FilterLaunch L{};
  L.a = *a;
  if (launch_filter(L, stream) != cudaSuccess) return PSPEC_ERR_CUDA;
  record_launches(1);
  return PSPEC_OK;
}

}  // extern "C"
