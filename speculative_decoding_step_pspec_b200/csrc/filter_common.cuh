// filter_common.cuh -- what the kernels of the filtered draw share: keys that order tokens, and a
// request's parameters made safe.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace pspec {

constexpr int kFilterSmallV = 2048;      // a row that a few warps hold in registers

__device__ __forceinline__ unsigned ord_of(float x) {       // order-preserving bits
  const unsigned b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
// Larger: the larger logit, of equal ones the lower id.
__device__ __forceinline__ unsigned long long key_of(float x, int id) {
  return (unsigned long long)ord_of(x) << 32 | (0xffffffffu - (unsigned)id);
}
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.f : -INFINITY; }  // NaN, -0

struct FilterParams {
  float temperature, top_p, min_p;
  long long k;
  bool k_on, p_on, m_on;
};

__device__ __forceinline__ FilterParams filter_params(const pspec_filter_args& a, long long seq, bool report) {
  FilterParams x;
  x.temperature = a.temperature ? __ldg(a.temperature + seq) : 1.f;
  x.top_p = a.top_p ? __ldg(a.top_p + seq) : 1.f;
  x.min_p = a.min_p ? __ldg(a.min_p + seq) : 0.f;
  x.k = a.top_k ? __ldg(a.top_k + seq) : 0;
  int bits = 0;
  if (!(x.temperature >= 0.f) || x.temperature == INFINITY) { x.temperature = 1.f; bits = PSPEC_DEVERR_PARAM_RANGE; }
  if (x.top_p != x.top_p) { x.top_p = 1.f; bits = PSPEC_DEVERR_PARAM_RANGE; }
  if (x.min_p != x.min_p) { x.min_p = 0.f; bits = PSPEC_DEVERR_PARAM_RANGE; }
  if (report) set_err(a.err, bits);
  if (x.min_p > 1.f || x.top_p <= 0.f) x.k = 1;             // only the first token is left
  if (x.top_p <= 0.f) x.top_p = 1.f;
  x.k_on = x.k > 0 && x.k < a.V;
  x.p_on = x.top_p < 1.f;
  x.m_on = x.min_p > 0.f && x.min_p <= 1.f;
  return x;
}

}  // namespace pspec
