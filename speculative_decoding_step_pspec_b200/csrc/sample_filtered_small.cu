// sample_filtered_small.cu -- the filtered draw over a small vocabulary (one launch).
//
// A team of 32 to 256 threads holds a row in registers, each thread consecutive tokens.  The
// largest key is the argmax; the cut of top-k and top-p is found on a sorted copy of the keys; the
// inverse CDF runs over the tokens as they lie, in id order.  Masses are fp64 as in the kernel
// for large vocabularies.  Teams of one warp share a CTA: rows of a few tokens cost what it takes
// to start them (3248 rows of 17 tokens, top-p: 8 us; by the kernel for large vocabularies: 234).
// Measured, mixed filters: 8192 rows of 20, 100, 500 and 2000 bf16 tokens 11, 24, 105 and 561 us;
// the sorting network's and the exponentials' instructions bound the longer ones.
#include "filter_common.cuh"

namespace pspec {

namespace {

template <int kT>
struct TeamSmem {
  double red[kT / 32];
  unsigned long long redk[kT / 32];
  unsigned long long cut;
  int first, last;
};

template <int kT>
struct Team {
  TeamSmem<kT>& sm;
  unsigned long long* keys;        // [kT * per] for the sort's far exchanges (kT > 32)
  int tid, lane, warp;

  __device__ __forceinline__ void sync() const {
    if constexpr (kT == 32) __syncwarp();
    else __syncthreads();
  }
  __device__ __forceinline__ unsigned long long max_key(unsigned long long k) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long x = __shfl_xor_sync(0xffffffffu, k, o);
      k = x > k ? x : k;
    }
    if constexpr (kT > 32) {
      sync();
      if (lane == 0) sm.redk[warp] = k;
      sync();
#pragma unroll
      for (int w = 0; w < kT / 32; ++w) k = sm.redk[w] > k ? sm.redk[w] : k;
    }
    return k;
  }
  __device__ __forceinline__ int total(int v) const {
    v = __reduce_add_sync(0xffffffffu, v);
    if constexpr (kT > 32) {
      sync();
      if (lane == 0) sm.redk[warp] = (unsigned)v;
      sync();
      v = 0;
#pragma unroll
      for (int w = 0; w < kT / 32; ++w) v += (int)sm.redk[w];
    }
    return v;
  }
  // Exclusive prefix of v over the threads, total in `all`.
  __device__ __forceinline__ double scan(double v, double& all) const {
    double inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += n;
    }
    if constexpr (kT == 32) {
      all = __shfl_sync(0xffffffffu, inc, 31);
      return inc - v;
    } else {
      sync();
      if (lane == 31) sm.red[warp] = inc;
      sync();
      double base = 0.0;
      all = 0.0;
#pragma unroll
      for (int w = 0; w < kT / 32; ++w) {
        if (w < warp) base += sm.red[w];
        all += sm.red[w];
      }
      return base + inc - v;
    }
  }
  // Keys descending, kPer consecutive ranks to a thread: a bitonic network.
  template <int kPer>
  __device__ __forceinline__ void sort(unsigned long long (&key)[kPer]) const {
    for (int k = 2; k <= kT * kPer; k <<= 1)
      for (int j = k >> 1; j > 0; j >>= 1) {
        if (kT > 32 && j >= 32 * kPer) {
          sync();
#pragma unroll
          for (int r = 0; r < kPer; ++r) keys[r * kT + tid] = key[r];
          sync();
        }
        if (j >= kPer) {
#pragma unroll
          for (int r = 0; r < kPer; ++r) {
            const unsigned long long o = kT > 32 && j >= 32 * kPer ? keys[r * kT + (tid ^ (j / kPer))]
                                                                   : __shfl_xor_sync(0xffffffffu, key[r], j / kPer);
            const int i = tid * kPer + r;
            key[r] = (((i & k) == 0) == ((i & j) == 0)) == (key[r] > o) ? key[r] : o;
          }
        } else {
#pragma unroll
          for (int jj = kPer / 2; jj > 0; jj >>= 1)
            if (jj == j) {
#pragma unroll
              for (int r = 0; r < kPer; ++r)
                if ((r & jj) == 0) {
                  const bool down = ((tid * kPer + r) & k) == 0;
                  const unsigned long long x = key[r], y = key[r + jj];
                  const bool swap = down ? x < y : x > y;
                  key[r] = swap ? y : x;
                  key[r + jj] = swap ? x : y;
                }
            }
        }
      }
  }
};

template <typename Tag, int kT, int kPer>
__global__ void __launch_bounds__(kT == 32 ? 128 : kT) filter_small_kernel(const FilterLaunch L) {
  constexpr int kTeams = kT == 32 ? 4 : 1;
  using elem = typename Tag::elem;
  __shared__ TeamSmem<kT> s_team[kTeams];
  __shared__ unsigned long long s_keys[kT == 32 ? 1 : kT * kPer];
  const pspec_filter_args& a = L.a;
  const int team = threadIdx.x / kT;
  const long long at = (long long)blockIdx.x * kTeams + team;
  if (at >= (long long)a.B * a.K) return;                   // (whole teams leave)
  const Team<kT> T{s_team[team], s_keys, (int)threadIdx.x % kT, (int)threadIdx.x & 31, (int)(threadIdx.x % kT) >> 5};
  const elem* row = static_cast<const elem*>(a.logits) + at * a.ld;
  const FilterParams prm = filter_params(a, at / a.K, T.tid == 0);
  const double u = (double)__ldg(a.uniforms + at);

  float x[kPer];
  unsigned long long key[kPer], best = 0;
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    const int id = T.tid * kPer + r;
    x[r] = id < a.V ? clean(load_scalar(row, id)) : -INFINITY;
    key[r] = x[r] > -INFINITY ? key_of(x[r], id) : 0;       // others are never kept
    best = key[r] > best ? key[r] : best;
  }
  best = T.max_key(best);
  auto write = [&](int token, double p) {
    a.tokens[at] = token;
    if (a.probs) a.probs[at] = (float)p;
  };
  if (best == 0 || prm.temperature == 0.f) {                // no mass: token 0; or the argmax
    if (T.tid == 0) write(best == 0 ? 0 : (int)(0xffffffffu - (unsigned)best), best == 0 ? 0.0 : 1.0);
    return;
  }
  // weights: exp((x - M) / temperature); with an infinite M those that equal it share the mass
  const float M = value_of((unsigned)(best >> 32));
  const double per = 1.0 / (double)prm.temperature;
  auto weight = [&](float v) { return v == M ? 1.0 : exp(((double)v - (double)M) * per); };
  unsigned long long cut = 0;
  if (prm.k_on || prm.p_on) {
    unsigned long long s[kPer];
#pragma unroll
    for (int r = 0; r < kPer; ++r) s[r] = key[r];
    T.template sort<kPer>(s);
    double w[kPer], sum = 0.0, all;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      const bool in = s[r] != 0 && (!prm.k_on || T.tid * kPer + r < prm.k);
      w[r] = in ? weight(value_of((unsigned)(s[r] >> 32))) : -1.0;
      sum += in ? w[r] : 0.0;
    }
    double mass = T.scan(sum, all);
    const double P = prm.p_on ? (double)prm.top_p * all : INFINITY;
    int kept = 0;                                           // a prefix: its length
#pragma unroll
    for (int r = 0; r < kPer; ++r)
      if (w[r] >= 0.0) {
        kept += mass < P;
        mass += w[r];
      }
    const int m = max(1, T.total(kept));
#pragma unroll
    for (int r = 0; r < kPer; ++r)
      if (T.tid * kPer + r == m - 1) T.sm.cut = s[r];
    T.sync();
    cut = T.sm.cut;
  }
  double w[kPer], sum = 0.0, all;
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    w[r] = key[r] != 0 && key[r] >= cut ? weight(x[r]) : 0.0;
    if (prm.m_on && w[r] < (double)prm.min_p) w[r] = 0.0;
    sum += w[r];
  }
  double mass = T.scan(sum, all);
  const double thr = u * all;
  int first = kNoIndex, last = -1;
#pragma unroll
  for (int r = 0; r < kPer; ++r) {
    mass += w[r];
    if (w[r] > 0.0) {
      last = T.tid * kPer + r;
      if (mass > thr) first = min(first, last);
    }
  }
  first = __reduce_min_sync(0xffffffffu, first);
  last = __reduce_max_sync(0xffffffffu, last);
  if constexpr (kT > 32) {
    if (T.tid == 0) {
      T.sm.first = kNoIndex;
      T.sm.last = -1;
    }
    T.sync();
    if (T.lane == 0) {
      atomicMin(&T.sm.first, first);
      atomicMax(&T.sm.last, last);
    }
    T.sync();
    first = T.sm.first;
    last = T.sm.last;
  }
  const int token = first != kNoIndex ? first : last;
#pragma unroll
  for (int r = 0; r < kPer; ++r)
    if (T.tid * kPer + r == token) write(token, w[r] / all);
}

template <typename Tag>
void launch_small(const FilterLaunch& L, cudaStream_t stream) {
  const long long rows = (long long)L.a.B * L.a.K;
  const unsigned by_warps = (unsigned)((rows + 3) / 4);
  const int V = L.a.V;
  if (V <= 32) filter_small_kernel<Tag, 32, 1><<<by_warps, 128, 0, stream>>>(L);
  else if (V <= 128) filter_small_kernel<Tag, 32, 4><<<by_warps, 128, 0, stream>>>(L);
  else if (V <= 512) filter_small_kernel<Tag, 128, 4><<<(unsigned)rows, 128, 0, stream>>>(L);
  else filter_small_kernel<Tag, 256, 8><<<(unsigned)rows, 256, 0, stream>>>(L);
}

}  // namespace

cudaError_t launch_filter_small(const FilterLaunch& L, cudaStream_t stream) {
  if (L.a.dtype == PSPEC_BF16) launch_small<BF16Tag>(L, stream);
  else launch_small<F32Tag>(L, stream);
  return cudaGetLastError();
}

}  // namespace pspec
