// sample_filtered.cu -- a token per row under temperature, top-k, top-p and min-p (one launch).
//
// Every filter keeps a prefix of the order (logit descending, id ascending), so what is kept is
// "all tokens up to one cut" and the cut is a 64-bit key: the logit's order-preserving bits
// above the inverted id.  A cluster of CTAs takes a row: each CTA copies its slice of the row
// into shared memory (the row is read from HBM once) and all later passes run there.
//   1. the row's maximum and smallest finite value;
//   2. top-k, then top-p: the bracket of keys that holds the cut is narrowed eight ways a pass
//      (count and mass of each part), until what is left fits into one CTA, which sorts it; when
//      everything above the bracket fits too, that CTA finishes the row alone;
//   3. else the masses of the kept tokens per chunk of 256, and the inverse CDF along them.
// Masses are fp64 sums of fp64 exponentials: the tokens drawn are compared with an exact draw,
// and with 10^5 tokens kept every 10^-8 of error in the running mass would change one row in a
// thousand.  Thread-private sums joined in a fixed order keep the results deterministic.
#include "common.cuh"
#include "kernels.h"

namespace pspec {

namespace {

constexpr int kFT = 512;                 // threads of a CTA
constexpr int kFW = kFT / 32;
constexpr int kWays = 8;                 // parts of the bracket per pass
constexpr int kGather = 2048;            // tokens that one CTA sorts
constexpr int kChunk = 256;              // 32 lanes x 8 elements
constexpr int kMaxCluster = 16;
constexpr size_t kSliceBytes = 128 * 1024;   // a slice above this is read from global memory

__device__ __forceinline__ unsigned ord_of(float x) {       // order-preserving bits
  const unsigned b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ unsigned long long key_of(float x, int id) {
  return (unsigned long long)ord_of(x) << 32 | (0xffffffffu - (unsigned)id);
}
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.f : -INFINITY; }  // NaN, -0

struct Part {            // what a CTA reports of one part of the bracket
  double mass;
  long long count;
};

struct FilterSmem {
  double table[32];                       // 2^(j/32)
  union {
    struct {
      double mass[kWays][kFT];
      int count[kWays][kFT];
    } col;
    struct {
      unsigned long long key[kGather];
      double w[kGather];
    } sort;
  };
  Part xch[2][kMaxCluster][kWays];        // exchange buffers, used in turn
  Part sum[kWays];
  double red[kFW];
  long long redi[kFW];
  double scan_total;
  unsigned long long cut;
  int gathered;
  int found, last;
};

__device__ __forceinline__ uint32_t cluster_map(const void* p, int rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_store(uint32_t a, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ int cluster_rank() {
  int r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

// 2^(y / 32) for y <= 0 in units of 1/32: 2^k * table[j] * e^f with f = (y - n) ln2 / 32, |f| <=
// 0.011, e^f by its Taylor polynomial of degree 5 (remainder below 3e-15).
__device__ __forceinline__ double exp2_32(double y, const double* table) {
  const double t = y + 6755399441055744.0;                  // 1.5 * 2^52: rounds to an integer
  const int n = __double2loint(t);
  const double f = (y - (t - 6755399441055744.0)) * 0.021660849392498290;
  double p = fma(f, 1.0 / 120.0, 1.0 / 24.0);
  p = fma(f, p, 1.0 / 6.0);
  p = fma(f, p, 0.5);
  p = fma(f, p, 1.0);
  p = fma(f, p, 1.0);
  p *= table[n & 31];
  return __hiloint2double(__double2hiint(p) + ((n >> 5) << 20), __double2loint(p));
}

template <typename Tag>
struct Filter {
  using elem = typename Tag::elem;
  FilterSmem& sm;
  const FilterLaunch& L;
  const elem* row;           // the row in global memory
  const elem* slice;         // this CTA's chunks: in shared memory, or the row's own
  double* chunk;             // [chunks of a CTA] kept mass
  bool vec;                  // slice starts on 16 bytes and is padded to whole chunks
  int V, G, rank, tid, lane, warp;
  int c0, nc;                // this CTA's chunks [c0, c0 + nc)
  int turn = 0;              // exchange buffer
  float M;
  double c32;                // 32 log2(e) / temperature
  double min_w;              // min_p, or 0

  __device__ Filter(FilterSmem& s, const FilterLaunch& l) : sm(s), L(l) {}

  __device__ double weight(float x) const {
    if (x == M) return 1.0;
    const double y = ((double)x - (double)M) * c32;
    return y < -32000.0 ? 0.0 : exp2_32(y, sm.table);       // y is NaN for no x here
  }

  // elements 8 lane .. 8 lane + 7 of local chunk c
  __device__ __forceinline__ void get8(int c, float (&x)[8]) const {
    const long long e = (long long)c * kChunk + lane * 8;
    if (vec) {
      if constexpr (sizeof(elem) == 2) {
        unpack(*reinterpret_cast<const uint4*>(slice + e), x, BF16Tag{});
      } else {
        const float4 a = *reinterpret_cast<const float4*>(slice + e);
        const float4 b = *reinterpret_cast<const float4*>(slice + e + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = (long long)c0 * kChunk + e + j < V ? load_scalar(slice, e + j) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = clean(x[j]);
  }
  __device__ __forceinline__ int id_of(int c, int j) const { return (c0 + c) * kChunk + lane * 8 + j; }

  // Every CTA's `n` parts sm.sum[0..n) to every CTA; all get them in rank order in the returned
  // buffer.  One cluster barrier.
  __device__ const Part (*exchange(int n))[kWays] {
    Part(*buf)[kWays] = sm.xch[turn];
    turn ^= 1;
    __syncthreads();
    for (int i = tid; i < G * n; i += kFT) {
      const int to = i / n, b = i - to * n;
      const uint32_t a = cluster_map(&buf[rank][b], to);
      cluster_store(a, (unsigned long long)__double_as_longlong(sm.sum[b].mass));
      cluster_store(a + 8, (unsigned long long)sm.sum[b].count);
    }
    cluster_sync();
    return buf;
  }

  __device__ double block_sum(double v) {                   // to every thread, fixed order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) sm.red[warp] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kFW; ++w) s += sm.red[w];
    return s;
  }

  // Exclusive prefix of v over the threads, total in `all`.
  __device__ double block_scan(double v, double& all) {
    double inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += n;
    }
    __syncthreads();
    if (lane == 31) sm.red[warp] = inc;
    __syncthreads();
    double base = 0.0;
    all = 0.0;
#pragma unroll
    for (int w = 0; w < kFW; ++w) {
      if (w < warp) base += sm.red[w];
      all += sm.red[w];
    }
    return base + inc - v;
  }

  // Mass of the tokens with key >= cut and weight >= min_w, per chunk into chunk[]; returns the
  // row's, and the mass of the CTAs before this one.
  __device__ double masses(unsigned long long cut, double& before) {
    const unsigned oc = (unsigned)(cut >> 32);
    double tot = 0.0;
    for (int c = warp; c < nc; c += kFW) {
      float x[8];
      get8(c, x);
      double s = 0.0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const unsigned o = ord_of(x[j]);
        if (o > oc || (o == oc && key_of(x[j], id_of(c, j)) >= cut)) {
          const double w = weight(x[j]);
          if (w >= min_w) s += w;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) chunk[c] = s;
      tot += s;
    }
    const double mine = block_sum(lane == 0 ? tot : 0.0);
    if (tid == 0) sm.sum[0] = Part{mine, 0};
    const Part(*all)[kWays] = exchange(1);
    double z = 0.0;
    before = 0.0;
    for (int r = 0; r < G; ++r) {
      if (r == rank) before = z;
      z += all[r][0].mass;
    }
    return z;
  }

  // sort.key[0, n) descending (ascending when up); n is padded to a power of two by the caller
  __device__ void bitonic(int n, bool up) {
    for (int k = 2; k <= n; k <<= 1)
      for (int j = k >> 1; j > 0; j >>= 1) {
        __syncthreads();
        for (int i = tid; i < n; i += kFT) {
          const int o = i ^ j;
          if (o > i) {
            const unsigned long long a = sm.sort.key[i], b = sm.sort.key[o];
            const bool down = ((i & k) == 0) != up;
            if (down ? a < b : a > b) {
              sm.sort.key[i] = b;
              sm.sort.key[o] = a;
              const double w = sm.sort.w[i];
              sm.sort.w[i] = sm.sort.w[o];
              sm.sort.w[o] = w;
            }
          }
        }
      }
    __syncthreads();
  }

  __device__ void write(int token, double p) {              // one thread
    const long long at = blockIdx.x / G;
    L.a.tokens[at] = token;
    if (L.a.probs) L.a.probs[at] = (float)p;
  }

  // The draw from kept tokens that lie in sort.key / sort.w [0, n), in any order (CTA 0 alone).
  __device__ void draw_gathered(int n, double u) {
    int pad = 1;
    while (pad < n) pad <<= 1;
    for (int i = tid; i < pad; i += kFT)
      sm.sort.key[i] = i < n ? 0xffffffffu - (sm.sort.key[i] & 0xffffffffull) : ~0ull;   // the id
    if (tid == 0) {
      sm.found = 0x7fffffff;
      sm.last = -1;
    }
    for (int i = n + tid; i < pad; i += kFT) sm.sort.w[i] = 0.0;
    bitonic(pad, true);
    constexpr int kPer = kGather / kFT;
    double w[kPer], s = 0.0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid * kPer + j;
      w[j] = i < n ? sm.sort.w[i] : 0.0;
      s += w[j];
    }
    double all;
    double at = block_scan(s, all);
    const double thr = u * all;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      at += w[j];
      if (w[j] > 0.0) {
        atomicMax(&sm.last, tid * kPer + j);
        if (at > thr) atomicMin(&sm.found, tid * kPer + j);
      }
    }
    __syncthreads();
    if (tid == 0) {
      const int i = sm.found != 0x7fffffff ? sm.found : sm.last;
      write((int)sm.sort.key[i], sm.sort.w[i] / all);
    }
  }

  // Narrows to the cut under "rank < k" and "mass before < P" among the tokens with key >= *cut.
  // `need_mass`: P is a limit.  Returns true when the row is finished (CTA 0 drew its token).
  // lo: no token with ord <= lo is kept for sure.
  __device__ bool select(unsigned long long* cut, long long k, double P, bool need_mass, unsigned lo,
                         float lowest, double top_p, bool top_p_after, double u) {
    unsigned hi = ord_of(M);
    const unsigned oc = (unsigned)(*cut >> 32);
    if (oc > 0 && oc - 1 > lo) lo = oc - 1;
    double above = 0.0;
    long long n_above = 0, n_in = V;
    bool exact_in = false;                                  // n_in counts the bracket's tokens
    for (int pass = 0;; ++pass) {
      const bool all_fit = n_above + n_in <= kGather;
      if (all_fit || (exact_in && (n_in <= kGather || hi - lo == 1))) {
        if (!all_fit && n_in > kGather) return tie(cut, hi, k - n_above, (P - above), n_in, need_mass);
        return finish(cut, k, P, need_mass, lo, all_fit ? 0xffffffffu : hi, all_fit ? 0.0 : above,
                      all_fit ? 0 : n_above, all_fit, top_p, top_p_after, u);
      }
      // parts (e[b+1], e[b]] of the bracket: equal in value, every other pass in key bits
      unsigned e[kWays + 1];
      e[0] = hi;
      e[kWays] = lo;
      const float vh = value_of(hi), vl = fmaxf(lo ? value_of(lo) : -INFINITY, lowest);
      const bool by_value = !(pass & 1) && vh - vl > 0.f && vh - vl < INFINITY;
#pragma unroll
      for (int b = 1; b < kWays; ++b) {
        unsigned o;
        if (by_value) o = ord_of(vh - (vh - vl) * ((float)b / kWays));
        else o = hi - (unsigned)((unsigned long long)(hi - lo) * b / kWays);
        e[b] = min(max(o, lo), b == 1 ? hi - 1 : e[b - 1]);    // part 0 holds hi itself
      }
      double* mass = &sm.col.mass[0][tid];
      int* count = &sm.col.count[0][tid];
      __syncthreads();
#pragma unroll
      for (int b = 0; b < kWays; ++b) {
        mass[b * kFT] = 0.0;
        count[b * kFT] = 0;
      }
      for (int c = warp; c < nc; c += kFW) {
        float x[8];
        get8(c, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const unsigned o = ord_of(x[j]);
          if (o > lo && o <= hi && id_of(c, j) < V && (o > oc || key_of(x[j], id_of(c, j)) >= *cut)) {
            int b = 0;
#pragma unroll
            for (int i = 1; i < kWays; ++i) b += o <= e[i];
            count[b * kFT] += 1;
            if (need_mass) mass[b * kFT] += weight(x[j]);
          }
        }
      }
      __syncthreads();
      if (warp < kWays) {
        double s = 0.0;
        long long n = 0;
        for (int i = lane; i < kFT; i += 32) {
          s += sm.col.mass[warp][i];
          n += sm.col.count[warp][i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          s += __shfl_xor_sync(0xffffffffu, s, o);
          n += __shfl_xor_sync(0xffffffffu, n, o);
        }
        if (lane == 0) sm.sum[warp] = Part{s, n};
      }
      const Part(*all)[kWays] = exchange(kWays);
      // the part that reaches a limit; the parts' masses add up to the bracket's only up to
      // rounding, so that none may: then the last part with tokens
      bool hit = false;
      Part run{above, n_above};
#pragma unroll
      for (int b = 0; b < kWays; ++b) {
        Part p{0.0, 0};
        for (int r = 0; r < G; ++r) {
          p.mass += all[r][b].mass;
          p.count += all[r][b].count;
        }
        if (!hit && p.count > 0) {
          hit = run.count + p.count >= k || (need_mass && run.mass + p.mass >= P);
          hi = e[b];
          lo = e[b + 1];
          n_in = p.count;
          n_above = run.count;
          above = run.mass;
        }
        run.mass += p.mass;
        run.count += p.count;
      }
      exact_in = true;
    }
  }

  // The bracket's tokens all have the same logit and are too many to sort: the first c of them
  // in id order are kept.
  __device__ bool tie(unsigned long long* cut, unsigned o, long long k_left, double P_left, long long n,
                      bool need_mass) {
    const double w = weight(value_of(o));
    long long c = min(n, k_left);
    if (need_mass && w > 0.0) {
      const double most = ceil(P_left / w);                 // token j is kept iff j w < P_left
      if (most < (double)c) c = max(1LL, (long long)most);
    }
    // the c-th tie: counts per chunk (as doubles: exact), then inside the chunk
    const unsigned long long old = *cut;
    double mine = 0.0;
    for (int ch = warp; ch < nc; ch += kFW) {
      float x[8];
      get8(ch, x);
      int m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        m += ord_of(x[j]) == o && id_of(ch, j) < V && key_of(x[j], id_of(ch, j)) >= old;
      m = __reduce_add_sync(0xffffffffu, m);
      if (lane == 0) chunk[ch] = m;
      mine += m;
    }
    const double tot = block_sum(lane == 0 ? mine : 0.0);
    if (tid == 0) {
      sm.sum[0] = Part{tot, 0};
      sm.cut = 0;
    }
    const Part(*all)[kWays] = exchange(1);
    double base = 0.0;
    for (int r = 0; r < rank; ++r) base += all[r][0].mass;
    if (base < (double)c && base + tot >= (double)c && warp == 0) {   // the c-th is here
      double at = base;
      int ch = 0;
      while (at + chunk[ch] < (double)c) at += chunk[ch++];
      float x[8];
      get8(ch, x);
      int m = 0;
      bool is[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        is[j] = ord_of(x[j]) == o && id_of(ch, j) < V && key_of(x[j], id_of(ch, j)) >= old;
        m += is[j];
      }
      int inc = m;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, s);
        if (lane >= s) inc += v;
      }
      int seen = (int)at - (int)base + inc - m;
      const int want = (int)((double)c - base);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (is[j] && ++seen == want)
          for (int r = 0; r < G; ++r) cluster_store(cluster_map(&sm.cut, r), key_of(x[j], id_of(ch, j)));
    }
    cluster_sync();
    *cut = sm.cut;
    return false;
  }

  // The tokens with lo < ord <= hi and key >= *cut go to CTA 0, which sorts them and finds the
  // cut; with `alone` they are all that can be kept, and it draws the token too.
  __device__ bool finish(unsigned long long* cut, long long k, double P, bool need_mass, unsigned lo,
                         unsigned hi, double above, long long n_above, bool alone, double top_p,
                         bool top_p_after, double u) {
    // CTA 0's counter starts at 0 and its sort arrays are free: the barrier before the copies
    __syncthreads();
    if (tid == 0) sm.gathered = 0;
    cluster_sync();
    const uint32_t counter = cluster_map(&sm.gathered, 0), keys = cluster_map(sm.sort.key, 0);
    for (int c = warp; c < nc; c += kFW) {
      float x[8];
      get8(c, x);
      unsigned in = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const unsigned o = ord_of(x[j]);
        if (o > lo && o <= hi && id_of(c, j) < V && key_of(x[j], id_of(c, j)) >= *cut) in |= 1u << j;
      }
      const int n = __popc(in);
      int inc = n;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, s);
        if (lane >= s) inc += v;
      }
      const int total = __shfl_sync(0xffffffffu, inc, 31);
      if (total == 0) continue;
      int at = 0;
      if (lane == 0)
        asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(at) : "r"(counter), "r"(total) : "memory");
      at = __shfl_sync(0xffffffffu, at, 0) + inc - n;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (in >> j & 1) {
          if (at < kGather) cluster_store(keys + 8 * at, key_of(x[j], id_of(c, j)));
          ++at;
        }
    }
    cluster_sync();
    if (rank == 0) {
      const int n = min(sm.gathered, kGather);
      int pad = 1;
      while (pad < n) pad <<= 1;
      for (int i = tid; i < pad; i += kFT) {
        if (i >= n) sm.sort.key[i] = 0;
        sm.sort.w[i] = i < n ? weight(value_of((unsigned)(sm.sort.key[i] >> 32))) : 0.0;
      }
      bitonic(pad, false);
      constexpr int kPer = kGather / kFT;
      double w[kPer], s = 0.0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = tid * kPer + j;
        w[j] = i < n && n_above + i < k ? sm.sort.w[i] : 0.0;   // the top-k set's masses
        s += w[j];
      }
      double all;
      double at = block_scan(s, all) + above;
      if (alone && top_p_after) {                           // top-p of the top-k set
        P = top_p * all;
        need_mass = true;
      }
      double kept = 0.0;                                    // a prefix: its length
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = tid * kPer + j;
        const bool in = i < n && n_above + i < k && (!need_mass || at < P) && (!alone || w[j] >= min_w);
        kept += in;
        at += w[j];
      }
      const int m = max(1, (int)block_sum(kept));
      if (alone) {
        draw_gathered(m, u);
      } else if (tid < G) {
        cluster_store(cluster_map(&sm.cut, tid), sm.sort.key[m - 1]);
      }
    }
    if (alone) return true;
    cluster_sync();
    *cut = sm.cut;
    return false;
  }

  // The token at u along the kept tokens' masses in id order.
  __device__ void draw(unsigned long long cut, double z, double before, double u) {
    // which CTA: the first whose running mass passes u z, else the last with mass
    const Part(*all)[kWays] = sm.xch[turn ^ 1];             // the exchange of masses()
    const double thr = u * z;
    int owner = -1, last = 0;
    double at = 0.0;
    for (int r = 0; r < G; ++r) {
      const double t = all[r][0].mass;
      at += t;
      if (t > 0.0) {
        last = r;
        if (owner < 0 && at > thr) owner = r;
      }
    }
    const bool crossing = owner >= 0;
    if (rank != (crossing ? owner : last)) return;
    if (tid == 0) {
      sm.found = 0x7fffffff;
      sm.last = -1;
    }
    __syncthreads();
    double base = before;
    int hit = -1;
    for (int c = 0; c < nc && hit < 0; c += kFT) {
      const double m = c + tid < nc ? chunk[c + tid] : 0.0;
      double sum;
      const double ex = block_scan(m, sum);
      if (m > 0.0) {
        atomicMax(&sm.last, c + tid);
        if (crossing && base + ex + m > thr) atomicMin(&sm.found, c + tid);
      }
      __syncthreads();
      if (sm.found != 0x7fffffff) {
        hit = sm.found;
        if (c + tid == hit) sm.scan_total = base + ex;
      }
      base += sum;
    }
    __syncthreads();
    const int ch = hit >= 0 ? hit : sm.last;
    if (warp == 0 && ch >= 0) {
      float x[8];
      double w[8], s = 0.0;
      get8(ch, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = key_of(x[j], id_of(ch, j)) >= cut ? weight(x[j]) : 0.0;
        if (w[j] < min_w) w[j] = 0.0;
        s += w[j];
      }
      double inc = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double n = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += n;
      }
      double run = (hit >= 0 ? sm.scan_total : 0.0) + inc - s;
      int first = 0x7fffffff, end = -1;
      double wf = 0.0, we = 0.0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        run += w[j];
        if (w[j] > 0.0) {
          end = lane * 8 + j;
          we = w[j];
          if (hit >= 0 && first == 0x7fffffff && run > thr) {
            first = end;
            wf = w[j];
          }
        }
      }
      const int f = __reduce_min_sync(0xffffffffu, first), l = __reduce_max_sync(0xffffffffu, end);
      const bool got = f != 0x7fffffff;
      if (got ? first == f : end == l) write((c0 + ch) * kChunk + (got ? f : l), (got ? wf : we) / z);
    }
  }
};

template <typename Tag>
__global__ void __launch_bounds__(kFT) filter_kernel(const FilterLaunch L) {
  using elem = typename Tag::elem;
  extern __shared__ __align__(16) uint8_t s_raw[];
  FilterSmem& sm = *reinterpret_cast<FilterSmem*>(s_raw);
  const pspec_filter_args& a = L.a;
  Filter<Tag> F(sm, L);
  F.V = a.V;
  F.G = L.cluster;
  F.rank = cluster_rank();
  F.tid = threadIdx.x;
  F.lane = threadIdx.x & 31;
  F.warp = threadIdx.x >> 5;
  const int tid = F.tid, lane = F.lane;
  const long long at = blockIdx.x / L.cluster;
  const long long seq = at / a.K;
  F.row = static_cast<const elem*>(a.logits) + at * a.ld;
  F.chunk = reinterpret_cast<double*>(s_raw + (sizeof(FilterSmem) + 15) / 16 * 16);
  const int chunks = (a.V + kChunk - 1) / kChunk;
  F.c0 = min(chunks, F.rank * L.chunks_per_cta);
  F.nc = min(chunks - F.c0, L.chunks_per_cta);

  if (tid < 32) sm.table[tid] = exp2((double)tid / 32.0);
  // ---- parameters
  float temp = a.temperature ? __ldg(a.temperature + seq) : 1.f;
  float top_p = a.top_p ? __ldg(a.top_p + seq) : 1.f;
  float min_p = a.min_p ? __ldg(a.min_p + seq) : 0.f;
  long long k = a.top_k ? __ldg(a.top_k + seq) : 0;
  const double u = (double)__ldg(a.uniforms + at);
  int bits = 0;
  if (!(temp >= 0.f) || temp == INFINITY) { temp = 1.f; bits = PSPEC_DEVERR_PARAM_RANGE; }
  if (top_p != top_p) { top_p = 1.f; bits = PSPEC_DEVERR_PARAM_RANGE; }
  if (min_p != min_p) { min_p = 0.f; bits = PSPEC_DEVERR_PARAM_RANGE; }
  if (F.rank == 0 && tid == 0) set_err(a.err, bits);
  if (min_p > 1.f || top_p <= 0.f) k = 1;                   // only the first token is left
  if (top_p <= 0.f) top_p = 1.f;
  const bool k_on = k > 0 && k < a.V, p_on = top_p < 1.f;
  F.min_w = min_p > 0.f && min_p <= 1.f ? (double)min_p : 0.0;
  F.c32 = temp > 0.f ? 32.0 * 1.4426950408889634074 / (double)temp : 0.0;

  // ---- the slice into shared memory, its largest and smallest finite values
  const long long e0 = (long long)F.c0 * kChunk;
  const int n = max(0, min(a.V - (int)min(e0, (long long)a.V), F.nc * kChunk));
  float hi = -INFINITY, lo = INFINITY;
  const elem* src = F.row + e0;
  if (L.resident) {
    elem* dst = reinterpret_cast<elem*>(F.chunk + (L.chunks_per_cta + 1) / 2 * 2);   // 16-byte aligned
    constexpr int W = Tag::kVec;
    const bool fast = (reinterpret_cast<uintptr_t>(src) & 15u) == 0;
    const int nv = fast ? n / W : 0;
    for (int i = tid; i < nv; i += kFT) {
      const uint4 v = ld_stream(src + (long long)i * W);
      float x[W];
      unpack(v, x, Tag{});
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float y = clean(x[j]);
        hi = fmaxf(hi, y);
        lo = fminf(lo, y == -INFINITY ? INFINITY : y);
      }
      *reinterpret_cast<uint4*>(dst + (long long)i * W) = v;
    }
    for (int i = nv * W + tid; i < F.nc * kChunk; i += kFT) {
      const float y = i < n ? clean(load_scalar(src, i)) : -INFINITY;
      hi = fmaxf(hi, y);
      lo = fminf(lo, y == -INFINITY ? INFINITY : y);
      if constexpr (sizeof(elem) == 2) dst[i] = (uint16_t)(__float_as_uint(y) >> 16);
      else dst[i] = y;
    }
    F.slice = dst;
    F.vec = true;
  } else {
    for (int i = tid; i < n; i += kFT) {
      const float y = clean(load_scalar(src, i));
      hi = fmaxf(hi, y);
      lo = fminf(lo, y == -INFINITY ? INFINITY : y);
    }
    F.slice = src;
    F.vec = false;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  if (lane == 0) {
    sm.red[F.warp] = hi;
    sm.redi[F.warp] = (long long)__float_as_int(lo);
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kFW; ++w) {
      hi = fmaxf(hi, (float)sm.red[w]);
      lo = fminf(lo, __int_as_float((int)sm.redi[w]));
    }
    sm.sum[0] = Part{(double)hi, (long long)__float_as_int(lo)};
  }
  cluster_sync();                                           // every CTA of the cluster runs
  {
    const Part(*all)[kWays] = F.exchange(1);
    F.M = -INFINITY;
    lo = INFINITY;
    for (int r = 0; r < F.G; ++r) {
      F.M = fmaxf(F.M, (float)all[r][0].mass);
      lo = fminf(lo, __int_as_float((int)all[r][0].count));
    }
  }
  if (F.M == -INFINITY) {                                   // no token has mass
    if (F.rank == 0 && tid == 0) F.write(0, 0.0);
    return;
  }
  if (temp == 0.f) {                                        // the argmax, lowest id
    int best = 0x7fffffff;
    for (int c = F.warp; c < F.nc; c += kFW) {
      float x[8];
      F.get8(c, x);
#pragma unroll
      for (int j = 7; j >= 0; --j)
        if (x[j] == F.M) best = min(best, F.id_of(c, j));
    }
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0) sm.redi[F.warp] = best;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kFW; ++w) best = min(best, (int)sm.redi[w]);
      sm.sum[0] = Part{0.0, best};
    }
    const Part(*all)[kWays] = F.exchange(1);
    for (int r = 0; r < F.G; ++r) best = min(best, (int)all[r][0].count);
    if (F.rank == 0 && tid == 0) F.write(best, 1.0);
    return;
  }

  unsigned long long cut = 0;
  const double min_w = F.min_w;
  double before;
  if (k_on && F.select(&cut, k, 0.0, false, 0u, lo, (double)top_p, p_on, u)) return;
  if (p_on) {
    F.min_w = 0.0;                                          // min-p does not enter top-p's mass
    const double z = F.masses(cut, before);
    F.min_w = min_w;
    // tokens lighter than (1 - p) z / V weigh less than (1 - p) z together: none is kept
    const double w0 = (1.0 - (double)top_p) * z / (double)a.V;
    const float floor_x = (float)((double)F.M + log2(w0) * 32.0 / F.c32);
    const float x0 = floor_x - fabsf(floor_x) * 1e-5f - 1e-30f;
    const unsigned lo_p = x0 > -INFINITY && x0 < F.M ? ord_of(x0) : 0u;
    if (F.select(&cut, 1LL << 40, (double)top_p * z, true, lo_p, lo, 1.0, false, u)) return;
  }
  const double z = F.masses(cut, before);
  F.draw(cut, z, before, u);
}

template <typename Tag>
cudaError_t launch_tag(FilterLaunch L, cudaStream_t stream) {
  const long long rows = (long long)L.a.B * L.a.K;
  const int chunks = (L.a.V + kChunk - 1) / kChunk;
  int G = 8;
  while (G > 1 && chunks < 2 * G) G >>= 1;
  L.cluster = G;
  L.chunks_per_cta = (chunks + G - 1) / G;
  const size_t slice = (size_t)L.chunks_per_cta * kChunk * sizeof(typename Tag::elem);
  L.resident = slice <= kSliceBytes;
  const size_t smem = (sizeof(FilterSmem) + 15) / 16 * 16 + (size_t)(L.chunks_per_cta + 1) / 2 * 16 +
                      (L.resident ? slice : 0);
  auto* fn = filter_kernel<Tag>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = G;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * G));
  cfg.blockDim = dim3(kFT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fn, L);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_filter(const FilterLaunch& L, cudaStream_t stream) {
  return L.a.dtype == PSPEC_BF16 ? launch_tag<BF16Tag>(L, stream) : launch_tag<F32Tag>(L, stream);
}

}  // namespace pspec
