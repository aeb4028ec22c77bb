// sample_filtered.cu -- a token per row under temperature, top-k, top-p and min-p (one launch).
//
// Every filter keeps a prefix of the order (logit descending, id ascending), so what is kept is
// "all tokens up to one cut" and the cut is a 64-bit key: the logit's order-preserving bits
// above the inverted id.  A cluster of CTAs takes a row: each CTA copies its slice of the row
// into shared memory (the row is read from HBM once) and all later passes run there.
//
// Two shortcuts keep those passes few.
//   A list: every thread keeps the largest logit that it loaded.  The R-th largest of these
//   maxima is a border with at least R tokens above it, and few more (tokens / threads of a row
//   are tens): the tokens above it go to one CTA, which sorts them.  With top-k (R = k) they
//   hold all that is kept; with top-p alone they do when their mass reaches p times the row's.
//   A bracket: for a nucleus longer than the list, passes over eight borders in fp32 close in on
//   the cut until the tokens between two of them fit the list; the mass above them is then summed
//   in fp64 and decides, so that fp32 is never part of an answer.
// Whatever these leave open (thousands of equal logits, top_k above kPick) is narrowed exactly,
// eight ways a pass on the keys' bits (`select`).
//
// Masses are fp64 sums of fp64 exponentials: the tokens drawn are compared with an exact draw,
// and with 10^5 tokens kept every 10^-8 of error in the running mass would change one row in a
// thousand.  Sums are joined in a fixed order, so results repeat.
#include "common.cuh"
#include "kernels.h"

namespace pspec {

namespace {

constexpr int kFT = 512;                 // threads of a CTA
constexpr int kFW = kFT / 32;
constexpr int kWays = 8;                 // parts of the bracket per pass
constexpr int kGather = 2048;            // tokens that one CTA sorts
constexpr int kPick = 1024;              // the largest rank looked for among the maxima
constexpr int kChunk = 256;              // 32 lanes x 8 elements
constexpr int kMaxCluster = 8;
constexpr size_t kSliceBytes = 128 * 1024;   // a slice above this is read from global memory
constexpr float kLowest = -3.402823466e38f;  // tokens below it (-inf) never have mass

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
// The key below those of every token with this value, above all smaller ones'.
__device__ __forceinline__ unsigned long long key_floor(float x) { return (unsigned long long)ord_of(x) << 32; }
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.f : -INFINITY; }  // NaN, -0

// The same on stored elements, eight (bf16) or four (fp32) at once; their maximum into `top`.
__device__ __forceinline__ uint32_t clean_pair(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b32 t;\n\tfma.rn.bf16x2 t, %1, %2, %3;\n\tmax.bf16x2 %0, t, %4;\n\t}"
      : "=r"(d) : "r"(w), "r"(0x3f803f80u), "r"(0u), "r"(0xff80ff80u));
  return d;
}
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void clean_vector(uint4& v, float& top, BF16Tag) {
  v.x = clean_pair(v.x); v.y = clean_pair(v.y); v.z = clean_pair(v.z); v.w = clean_pair(v.w);
  const uint32_t m = max_pair(max_pair(v.x, v.y), max_pair(v.z, v.w));
  top = fmaxf(top, fmaxf(bf16_lo(m), bf16_hi(m)));
}
__device__ __forceinline__ void clean_vector(uint4& v, float& top, F32Tag) {
  const float a = clean(__uint_as_float(v.x)), b = clean(__uint_as_float(v.y));
  const float c = clean(__uint_as_float(v.z)), d = clean(__uint_as_float(v.w));
  v = make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
  top = fmaxf(top, fmaxf(fmaxf(a, b), fmaxf(c, d)));
}
__device__ __forceinline__ uint16_t elem_of(float x, uint16_t) { return (uint16_t)(__float_as_uint(x) >> 16); }
__device__ __forceinline__ float elem_of(float x, float) { return x; }
__device__ __forceinline__ float load_generic(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float load_generic(const float* p) { return *p; }

struct Part {            // what a CTA reports of one part of the bracket
  double mass;
  long long count;
};

struct FilterSmem {
  double table[128];                      // 2^(j/128)
  union {
    unsigned long long key[kGather];
    unsigned top[kMaxCluster * kFT];      // CTA 0: the maxima of the cluster's threads
  };
  Part xch[2][kMaxCluster][kWays];        // exchange buffers, used in turn
  Part sum[kWays];
  double strip[kFW];                      // kept mass of each warp's strip
  double red[kFW];
  int redi[2][kFW];
  float part[kFW][kWays];
  double wide[kFW][kWays];
  int widei[kFW][kWays];
  unsigned long long cut;                 // CTA 0's answers to the cluster
  double mass;
  float pick;
  int ok;
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
__device__ __forceinline__ void cluster_store32(uint32_t a, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
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
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src));
}

template <typename Tag>
struct Filter {
  using elem = typename Tag::elem;
  FilterSmem& sm;
  const FilterLaunch& L;
  const elem* row;           // the row in global memory
  elem* slice;               // this CTA's chunks in shared memory (resident)
  int V, G, rank, tid, lane, warp;
  int lead;                  // the row is placed at this element of its first chunk, so that
                             // 16-byte aligned pieces of it are aligned in the slice too
  int c0, nc;                // this CTA's chunks [c0, c0 + nc)
  int turn = 0;              // exchange buffer
  bool resident;
  float M, zero_below;       // largest logit; tokens below the second weigh nothing
  double Md, c;              // M, and 128 log2(e) / temperature

  __device__ Filter(FilterSmem& s, const FilterLaunch& l) : sm(s), L(l) {}

  // exp((x - M) / temperature) = 2^(y/128), y = (x - M) c <= 0: 2^k * table[j] * e^g with
  // g = (y - n) ln2 / 128, |g| <= 0.0028, e^g by its Taylor polynomial of degree 3 (remainder
  // below 2.4e-12).  Tokens below zero_below (y < -128000) weigh nothing.
  __device__ __forceinline__ void factors(float x, double& scale, double& poly) const {
    constexpr double a = 0.69314718055994530942 / 128.0;
    const double d = (double)fmaxf(x, zero_below) - Md;
    const double t = fma(d, c, 6755399441055744.0);          // 1.5 * 2^52: rounds to an integer
    const int n = __double2loint(t);
    const double f = fma(d, c, 6755399441055744.0 - t);
    poly = fma(f, fma(f, fma(f, a * a * a / 6.0, a * a / 2.0), a), 1.0);
    const double b = sm.table[n & 127];
    scale = __hiloint2double(__double2hiint(b) + ((n >> 7) << 20), __double2loint(b));
    if (x < zero_below) scale = 0.0;
  }
  __device__ double weight(float x) const {
    double s, p;
    factors(x, s, p);
    return s * p;
  }

  // elements 8v .. 8v + 7 of the CTA's chunks; what lies outside the row is -inf
  __device__ __forceinline__ void get8(int v, float (&x)[8]) const {
    const long long e = (long long)v * 8;
    if (resident) {
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
      for (int j = 0; j < 8; ++j) {
        const int id = id_of(v, j);
        x[j] = id >= 0 && id < V ? clean(load_scalar(row, id)) : -INFINITY;
      }
      if (inf_row) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] == INFINITY ? 0.f : -INFINITY;
      }
    }
  }
  bool inf_row = false;      // the largest logit is +inf: those count as 0, all others as -inf
  __device__ __forceinline__ int id_of(int v, int j) const { return c0 * kChunk + v * 8 + j - lead; }

  // A warp's strip of the CTA's vectors of eight.
  __device__ __forceinline__ int strip_lo(int w) const { return (int)((long long)nc * 32 * w / kFW); }

  // f(v, x) for the eight elements of each of this lane's vectors, whole warps at a time.
  template <typename F>
  __device__ __forceinline__ void sweep(F&& f) const {
    const int lo = strip_lo(warp), hi = strip_lo(warp + 1);
    for (int v0 = lo; v0 < hi; v0 += 32) {
      float x[8];
      if (v0 + lane < hi) {
        get8(v0 + lane, x);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = -INFINITY;
      }
      f(v0 + lane, x);
    }
  }

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

  __device__ int block_count(int v, int slot) {             // alternate `slot` between calls
    v = __reduce_add_sync(0xffffffffu, v);
    if (lane == 0) sm.redi[slot][warp] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < kFW; ++w) s += sm.redi[slot][w];
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

  // Mass of the tokens with key >= cut (all: every token) by strips; returns the row's, and the
  // mass of the CTAs before this one.
  template <bool kAll>
  __device__ double masses(unsigned long long cut, double& before) {
    const float xc = kAll ? kLowest : value_of((unsigned)(cut >> 32));
    const unsigned low = (unsigned)cut;
    double a = 0.0;
    sweep([&](int v, const float (&x)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (kAll || x[j] > xc || (x[j] == xc && 0xffffffffu - (unsigned)id_of(v, j) >= low)) {
          double s, p;
          factors(x[j], s, p);
          a = fma(s, p, a);
        }
      }
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    __syncthreads();
    if (lane == 0) sm.strip[warp] = a;
    __syncthreads();
    if (tid == 0) {
      double s = 0.0;
      for (int w = 0; w < kFW; ++w) s += sm.strip[w];
      sm.sum[0] = Part{s, 0};
    }
    const Part(*all)[kWays] = exchange(1);
    double z = 0.0;
    before = 0.0;
    for (int r = 0; r < G; ++r) {
      if (r == rank) before = z;
      z += all[r][0].mass;
    }
    return z;
  }

  // Keys descending over the CTA, kPer to a thread (thread t holds the ranks kPer t ...): a
  // bitonic network, its close exchanges in registers and between lanes.
  template <int kPer>
  __device__ __forceinline__ void sort(unsigned long long (&key)[kPer]) {
    constexpr int N = kPer * kFT;
    for (int k = 2; k <= N; k <<= 1) {
      for (int j = k >> 1; j > 0; j >>= 1) {
        if (j >= 32 * kPer) {
          __syncthreads();
#pragma unroll
          for (int r = 0; r < kPer; ++r) sm.key[r * kFT + tid] = key[r];
          __syncthreads();
#pragma unroll
          for (int r = 0; r < kPer; ++r) {
            const unsigned long long o = sm.key[r * kFT + (tid ^ (j / kPer))];
            const int i = tid * kPer + r;
            key[r] = (((i & k) == 0) == ((i & j) == 0)) == (key[r] > o) ? key[r] : o;
          }
        } else if (j >= kPer) {
#pragma unroll
          for (int r = 0; r < kPer; ++r) {
            const unsigned long long o = __shfl_xor_sync(0xffffffffu, key[r], j / kPer);
            const int i = tid * kPer + r;
            key[r] = (((i & k) == 0) == ((i & j) == 0)) == (key[r] > o) ? key[r] : o;
          }
        } else {
#pragma unroll
          for (int jj = kPer / 2; jj > 0; jj >>= 1) {
            if (jj == j) {
#pragma unroll
              for (int r = 0; r < kPer; ++r)
                if ((r & jj) == 0) {
                  const bool down = ((tid * kPer + r) & k) == 0;
                  const unsigned long long a = key[r], b = key[r + jj];
                  const bool swap = down ? a < b : a > b;
                  key[r] = swap ? b : a;
                  key[r + jj] = swap ? a : b;
                }
            }
          }
        }
      }
    }
  }

  __device__ void write(int token, double p) {              // one thread
    const long long at = blockIdx.x / G;
    L.a.tokens[at] = token;
    if (L.a.probs) L.a.probs[at] = (float)p;
  }

  // ------------------------------------------------------------------ the list
  // The border: a value with at least R of the maxima, and few more, at or above it (kLowest
  // when fewer are finite).  CTA 0 looks, all get the answer.  Two cluster barriers at most; the
  // first one of the row must lie between the maxima's stores and this.
  __device__ float pick(int R) {
    if (rank == 0) {
      constexpr int kPer = kMaxCluster;
      float x[kPer];
      float least = INFINITY;
      int finite = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        x[i] = i < G ? __uint_as_float(sm.top[i * kFT + tid]) : -INFINITY;
        if (x[i] > -INFINITY) {
          least = fminf(least, x[i]);
          ++finite;
        }
      }
      // the smallest finite maximum, as an integer of the same order
      const unsigned o = __reduce_min_sync(0xffffffffu, ord_of(least));
      if (lane == 0) sm.redi[0][warp] = (int)o;
      __syncthreads();
      unsigned lo_o = 0xffffffffu;
      for (int w = 0; w < kFW; ++w) lo_o = min(lo_o, (unsigned)sm.redi[0][w]);
      float t = kLowest;
      if (block_count(finite, 1) >= R) {
        float lo = value_of(lo_o), hi = M;                  // count(>= lo) >= R
        t = lo;
        for (int step = 0; step < 24; ++step) {
          const float mid = 0.5f * lo + 0.5f * hi;
          if (!(mid > lo)) break;
          int n = 0;
#pragma unroll
          for (int i = 0; i < kPer; ++i) n += x[i] >= mid;
          n = block_count(n, step & 1);
          if (n >= R) {
            t = lo = mid;
            if (n <= R + R / 8 + 4) break;
          } else {
            if (mid == hi) break;
            hi = mid;
          }
        }
      }
      if (tid < G) cluster_store32(cluster_map(&sm.pick, tid), __float_as_uint(t));
    }
    cluster_sync();
    return sm.pick;
  }

  // The tokens with lo <= x < hi and key >= cut (hi: +inf for no limit; lo is not below the cut's
  // value) into CTA 0's keys, in no fixed order; returns how many, and copies nothing when they
  // are more than kGather.  Two cluster barriers.
  __device__ int gather(float lo, float hi, unsigned long long cut) {
    const unsigned low = value_of((unsigned)(cut >> 32)) == lo ? (unsigned)cut : 0u;
    __syncthreads();
    if (tid == 0) sm.gathered = 0;
    __syncthreads();
    sweep([&](int v, const float (&x)[8]) {
      unsigned in = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) in |= (x[j] >= lo && x[j] < hi ? 1u : 0u) << j;
      if (low != 0) {                                       // a cut inside the ties of its value
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (x[j] == lo && 0xffffffffu - (unsigned)id_of(v, j) < low) in &= ~(1u << j);
      }
      if (__any_sync(0xffffffffu, in != 0)) {
        const int n = __popc(in);
        int inc = n;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, inc, s);
          if (lane >= s) inc += o;
        }
        int at = 0;
        if (lane == 31) at = atomicAdd(&sm.gathered, inc);
        at = __shfl_sync(0xffffffffu, at, 31) + inc - n;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (in >> j & 1) {
            if (at < kGather) sm.key[at] = key_of(x[j], id_of(v, j));
            ++at;
          }
      }
    });
    __syncthreads();
    if (tid == 0) sm.sum[0] = Part{0.0, sm.gathered};
    const Part(*all)[kWays] = exchange(1);
    long long n = 0, off = 0;
    for (int r = 0; r < G; ++r) {
      if (r == rank) off = n;
      n += all[r][0].count;
    }
    if (n <= kGather) {
      if (rank > 0) {
        const int mine = (int)all[rank][0].count;
        const uint32_t to = cluster_map(sm.key, 0) + 8 * (uint32_t)off;
        for (int i = tid; i < mine; i += kFT) cluster_store(to + 8 * i, sm.key[i]);
      }
      cluster_sync();
    }
    return (int)min(n, (long long)kGather + 1);
  }

  // What CTA 0 makes of the n tokens in its keys.
  struct List {
    long long k;             // ranks below k are kept (of the whole row: n_above lie above the list)
    long long n_above;
    double above;            // mass above the list
    double P;                // mass before a kept token is below P (INFINITY: off) ...
    double top_p;            // ... or below top_p times the top-k set's mass (< 1: on)
    float min_x;             // smallest value that min-p keeps
    bool draw;               // draw the token (nothing is above the list)
    bool reach;              // the list must reach P, else it answers "not here"
  };
  // With `reach` or without `draw`, whether the list held the cut, the cut and the list's mass go
  // to every CTA's sm.ok, sm.cut and sm.mass, and the cluster barrier is arrived at.
  template <int kPer>
  __device__ void settle(int n, List q, double u) {
    unsigned long long key[kPer];
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      const int i = r * kFT + tid;                          // any order will do
      key[r] = i < n ? sm.key[i] : 0;
    }
    sort<kPer>(key);
    double w[kPer], s = 0.0;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      const int i = tid * kPer + r;
      w[r] = i < n && q.n_above + i < q.k ? weight(value_of((unsigned)(key[r] >> 32))) : 0.0;
      s += w[r];
    }
    double all;
    double at = block_scan(s, all) + q.above;
    if (q.top_p < 1.0) q.P = q.top_p * all;
    const bool ok = !q.reach || (q.above < q.P && q.above + all >= q.P);
    int kept = 0;                                           // a prefix: its length
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      const int i = tid * kPer + r;
      kept += i < n && q.n_above + i < q.k && at < q.P && value_of((unsigned)(key[r] >> 32)) >= q.min_x;
      at += w[r];
    }
    __syncthreads();
    const int m = max(1, block_count(kept, 0));
    if (q.reach || !q.draw) {
#pragma unroll
      for (int r = 0; r < kPer; ++r)
        if (tid * kPer + r == m - 1)
          for (int g = 0; g < G; ++g) cluster_store(cluster_map(&sm.cut, g), key[r]);
      if (tid < G) {
        cluster_store(cluster_map(&sm.mass, tid), (unsigned long long)__double_as_longlong(all));
        cluster_store32(cluster_map(&sm.ok, tid), ok);
      }
      cluster_arrive();
    }
    if (!ok || !q.draw) return;
    // the kept tokens in id order: sorted by the inverted id, which is the keys' low half
#pragma unroll
    for (int r = 0; r < kPer; ++r)
      key[r] = tid * kPer + r < m ? key[r] << 32 | key[r] >> 32 : 0;
    sort<kPer>(key);
    s = 0.0;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      w[r] = tid * kPer + r < m ? weight(value_of((unsigned)key[r])) : 0.0;
      s += w[r];
    }
    if (tid == 0) {
      sm.found = kNoIndex;
      sm.last = -1;
    }
    at = block_scan(s, all);
    const double thr = u * all;
    int first = kNoIndex, end = -1;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      at += w[r];
      if (w[r] > 0.0) {
        end = tid * kPer + r;
        if (at > thr) first = min(first, end);
      }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    end = __reduce_max_sync(0xffffffffu, end);
    if (lane == 0) {
      if (first != kNoIndex) atomicMin(&sm.found, first);
      if (end >= 0) atomicMax(&sm.last, end);
    }
    __syncthreads();
    const int i = sm.found != kNoIndex ? sm.found : sm.last;
#pragma unroll
    for (int r = 0; r < kPer; ++r)
      if (tid * kPer + r == i) write((int)(0xffffffffu - (unsigned)(key[r] >> 32)), w[r] / all);
  }
  // Every CTA calls this; returns sm.ok (true when the token is drawn without `reach`).
  __device__ bool settle(int n, const List& q, double u) {
    const bool answer = q.reach || !q.draw;
    if (rank == 0) {
      if (n <= kFT) settle<1>(n, q, u);
      else settle<kGather / kFT>(n, q, u);
    } else if (answer) {
      cluster_arrive();
    }
    if (!answer) return true;
    cluster_wait();
    return sm.ok != 0;
  }

  // ------------------------------------------------------------------ the bracket
  // Closes [lo, hi) in on the value at which the mass above passes P, given the mass A above hi;
  // fp32 sums, an answer to be verified.  False when it does not come down to a list.
  __device__ bool narrow(float& lo, float& hi, double A, double P) {
    const float cf = (float)(c / 128.0);
    for (int pass = 0; pass < 6; ++pass) {
      const float span = hi - lo;
      if (!(span > 0.f) || !(span < INFINITY)) return false;
      float e[kWays], acc[kWays];
#pragma unroll
      for (int i = 0; i < kWays; ++i) {
        e[i] = i + 1 < kWays ? hi - span * ((float)(i + 1) / kWays) : lo;
        acc[i] = 0.f;
      }
      sweep([&](int, const float (&x)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float w = x[j] < hi ? ex2((x[j] - M) * cf) : 0.f;
#pragma unroll
          for (int i = 0; i < kWays; ++i) acc[i] += x[j] >= e[i] ? w : 0.f;
        }
      });
#pragma unroll
      for (int i = 0; i < kWays; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      __syncthreads();
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kWays; ++i) sm.part[warp][i] = acc[i];
      }
      __syncthreads();
      if (tid < kWays) {
        double s = 0.0;
        for (int w = 0; w < kFW; ++w) s += sm.part[w][tid];
        sm.sum[tid] = Part{s, 0};
      }
      const Part(*all)[kWays] = exchange(kWays);
      double below = 0.0, upto = 0.0;                       // masses between hi and the new borders
      float new_hi = hi, new_lo = lo;
      bool past = false;
#pragma unroll
      for (int i = 0; i < kWays; ++i) {
        double s = 0.0;
        for (int r = 0; r < G; ++r) s += all[r][i].mass;
        if (i + 1 < kWays && A + s <= P * (1.0 - 1e-5)) {
          new_hi = e[i];
          below = s;
        }
        if (!past) {
          upto = s;
          new_lo = e[i];
          past = A + s >= P * (1.0 + 1e-5);
        }
      }
      hi = new_hi;
      lo = new_lo;
      A += below;
      // tokens of the bracket weigh at least what its lower border does
      if (upto - below <= (kGather - 100) * (double)ex2((lo - M) * cf)) return true;
    }
    return false;
  }

  // ------------------------------------------------------------------ exact narrowing
  // The cut under "rank < k" and "mass before < P" among the tokens with key >= old.
  // `need_mass`: P is a limit.
  __device__ unsigned long long select(unsigned long long old, long long k, double P, bool need_mass) {
    unsigned hi = ord_of(M), lo = ord_of(-INFINITY);
    const unsigned oc = (unsigned)(old >> 32);
    if (oc > 0 && oc - 1 > lo) lo = oc - 1;
    double above = 0.0;
    long long n_above = 0, n_in = 0;
    do {
      // parts (e[b+1], e[b]] of the bracket, equal in key bits
      unsigned e[kWays + 1];
      e[0] = hi;
      e[kWays] = lo;
#pragma unroll
      for (int b = 1; b < kWays; ++b) {
        const unsigned o = hi - (unsigned)((unsigned long long)(hi - lo) * b / kWays);
        e[b] = min(max(o, lo), b == 1 ? hi - 1 : e[b - 1]);    // part 0 holds hi itself
      }
      double mass[kWays];
      int count[kWays];
#pragma unroll
      for (int b = 0; b < kWays; ++b) {
        mass[b] = 0.0;
        count[b] = 0;
      }
      sweep([&](int v, const float (&x)[8]) {
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
          float y = x[0];
#pragma unroll
          for (int i = 1; i < 8; ++i) y = j == i ? x[i] : y;
          const unsigned o = ord_of(y);
          if (o > lo && o <= hi && (o > oc || key_of(y, id_of(v, j)) >= old)) {
            const double w = need_mass ? weight(y) : 0.0;
#pragma unroll
            for (int b = 0; b < kWays; ++b)
              if (o <= e[b] && o > e[b + 1]) {
                mass[b] += w;
                ++count[b];
              }
          }
        }
      });
      __syncthreads();
#pragma unroll
      for (int b = 0; b < kWays; ++b) {
        double s = mass[b];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const int n = __reduce_add_sync(0xffffffffu, count[b]);
        if (lane == 0) {
          sm.wide[warp][b] = s;
          sm.widei[warp][b] = n;
        }
      }
      __syncthreads();
      if (tid < kWays) {
        Part p{0.0, 0};
        for (int w = 0; w < kFW; ++w) {
          p.mass += sm.wide[w][tid];
          p.count += sm.widei[w][tid];
        }
        sm.sum[tid] = p;
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
    } while (n_in > kGather && hi - lo > 1);
    if (n_in > kGather) return tie(old, value_of(hi), k - n_above, P - above, n_in, need_mass);
    const int n = gather(value_of(lo + 1), value_of(hi + 1), old);
    List q{};
    q.k = k;
    q.n_above = n_above;
    q.above = above;
    q.P = need_mass ? P : INFINITY;
    q.top_p = 1.0;
    q.min_x = kLowest;
    settle(n, q, 0.0);
    return sm.cut;
  }

  // n tokens with logit x (among those with key >= old), too many to sort: the cut that keeps the
  // first ones in id order.
  __device__ unsigned long long tie(unsigned long long old, float xt, long long k_left, double P_left,
                                    long long n, bool need_mass) {
    const double w = weight(xt);
    long long c = min(n, k_left);
    if (need_mass && w > 0.0) {
      const double most = ceil(P_left / w);                 // token j is kept iff j w < P_left
      if (most < (double)c) c = max(1LL, (long long)most);
    }
    // the c-th tie: counts per strip (as doubles: exact), then inside the strip
    const float x_old = value_of((unsigned)(old >> 32));
    auto is_tie = [&](float x, int id) {
      return x == xt && (x > x_old || 0xffffffffu - (unsigned)id >= (unsigned)old);
    };
    int mine = 0;
    sweep([&](int v, const float (&x)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) mine += is_tie(x[j], id_of(v, j));
    });
    mine = __reduce_add_sync(0xffffffffu, mine);
    __syncthreads();
    if (lane == 0) sm.strip[warp] = mine;
    __syncthreads();
    if (tid == 0) {
      double s = 0.0;
      for (int i = 0; i < kFW; ++i) s += sm.strip[i];
      sm.sum[0] = Part{s, 0};
      sm.cut = 0;
    }
    const Part(*all)[kWays] = exchange(1);
    double base = 0.0;
    for (int r = 0; r < rank; ++r) base += all[r][0].mass;
    for (int i = 0; i < warp; ++i) base += sm.strip[i];
    if (base < (double)c && base + sm.strip[warp] >= (double)c) {      // the c-th is in this strip
      int seen = 0;
      const int want = (int)((double)c - base);
      sweep([&](int v, const float (&x)[8]) {
        unsigned is = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) is |= (is_tie(x[j], id_of(v, j)) ? 1u : 0u) << j;
        int inc = __popc(is);
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, inc, s);
          if (lane >= s) inc += o;
        }
        int at = seen + inc - __popc(is);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((is >> j & 1) && ++at == want)
            for (int r = 0; r < G; ++r) cluster_store(cluster_map(&sm.cut, r), key_of(x[j], id_of(v, j)));
        seen += __shfl_sync(0xffffffffu, inc, 31);
      });
    }
    cluster_sync();
    return sm.cut;
  }

  // ------------------------------------------------------------------ the draw along the row
  // The token at u along the kept tokens' masses in id order; after masses(cut).
  template <bool kAll>
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
    if (rank != (owner >= 0 ? owner : last)) return;
    // which strip, the same way
    double base = before, start = before;
    int strip = -1, end = 0;
    for (int i = 0; i < kFW; ++i) {
      const double t = sm.strip[i];
      if (t > 0.0) {
        if (strip < 0) start = base;
        end = i;
        if (strip < 0 && base + t > thr) strip = i;
      }
      base += t;
    }
    if (warp != (strip >= 0 ? strip : end)) return;
    // which token: the strip's vectors in turn
    const float xc = kAll ? kLowest : value_of((unsigned)(cut >> 32));
    const unsigned low = (unsigned)cut;
    double run = strip >= 0 ? start : -INFINITY;
    int first = kNoIndex, tail = -1;
    double wf = 0.0, wt = 0.0;
    sweep([&](int v, const float (&x)[8]) {
      if (first != kNoIndex) return;                        // the same in every lane
      double w[8], s = 0.0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = kAll || x[j] > xc || (x[j] == xc && 0xffffffffu - (unsigned)id_of(v, j) >= low);
        w[j] = in ? weight(x[j]) : 0.0;
        s += w[j];
      }
      double inc = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double n = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += n;
      }
      double r = run + inc - s;
      int f = kNoIndex, e = -1;
      double w_f = 0.0, w_e = 0.0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r += w[j];
        if (w[j] > 0.0) {
          e = id_of(v, j);
          w_e = w[j];
          if (f == kNoIndex && r > thr) {
            f = e;
            w_f = w[j];
          }
        }
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
      first = __reduce_min_sync(0xffffffffu, f);
      if (first == f) wf = w_f;
      const int t = __reduce_max_sync(0xffffffffu, e);
      if (t > tail) {
        tail = t;
        wt = e == t ? w_e : 0.0;
      }
    });
    if (first != kNoIndex) {
      if (wf > 0.0) write(first, wf / z);
    } else if (wt > 0.0) {
      write(tail, wt / z);
    }
  }
};

template <typename Tag>
__global__ void __launch_bounds__(kFT, 2) filter_kernel(const FilterLaunch L) {
  using elem = typename Tag::elem;
  constexpr int W = Tag::kVec;
  extern __shared__ __align__(16) uint8_t s_raw[];
  FilterSmem& sm = *reinterpret_cast<FilterSmem*>(s_raw);
  const pspec_filter_args& a = L.a;
  cluster_arrive();                                         // waited for before the first remote store
  Filter<Tag> F(sm, L);
  F.V = a.V;
  F.G = L.cluster;
  F.rank = cluster_rank();
  F.tid = threadIdx.x;
  F.lane = threadIdx.x & 31;
  F.warp = threadIdx.x >> 5;
  const int tid = F.tid, lane = F.lane, warp = F.warp;
  const long long at = blockIdx.x / L.cluster;
  const long long seq = at / a.K;
  F.row = static_cast<const elem*>(a.logits) + at * a.ld;
  F.resident = L.resident != 0;
  F.lead = F.resident ? (int)((reinterpret_cast<uintptr_t>(F.row) & 15u) / sizeof(elem)) : 0;
  const int chunks = (int)(((long long)a.V + F.lead + kChunk - 1) / kChunk);
  F.c0 = min(chunks, F.rank * L.chunks_per_cta);
  F.nc = min(chunks - F.c0, L.chunks_per_cta);
  const int n = F.nc * kChunk;                              // elements of the slice
  F.slice = reinterpret_cast<elem*>(s_raw + (sizeof(FilterSmem) + 15) / 16 * 16);

  // ---- the slice into shared memory: every thread its own 16-byte pieces, in flight together;
  // pieces at the row's ends by elements
  const int vectors = n / W, per = (vectors + kFT - 1) / kFT;
  if (F.resident) {
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(F.slice);
    const int id0 = F.c0 * kChunk - F.lead;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      for (int m = q * per / 4; m < (q + 1) * per / 4; ++m) {
        const int i = m * kFT + tid;
        const int id = id0 + i * W;
        if (i < vectors) {
          if (id >= 0 && id + W <= a.V) {
            copy16(dst + i * 16, F.row + id);
          } else {
            for (int j = 0; j < W; ++j)
              F.slice[i * W + j] = elem_of(id + j >= 0 && id + j < a.V ? load_scalar(F.row, id + j) : -INFINITY, elem{});
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }

  // ---- parameters
  if (tid < 128) sm.table[tid] = exp2((double)tid / 128.0);
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
  const bool k_on = k > 0 && k < a.V, p_on = top_p < 1.f, m_on = min_p > 0.f && min_p <= 1.f;

  // ---- NaN and -0 taken out, the thread's largest logit
  float top = -INFINITY;
  if (F.resident) {
    uint4* s = reinterpret_cast<uint4*>(F.slice);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q == 0) asm volatile("cp.async.wait_group 3;" ::: "memory");
      if (q == 1) asm volatile("cp.async.wait_group 2;" ::: "memory");
      if (q == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      if (q == 3) asm volatile("cp.async.wait_group 0;" ::: "memory");
      for (int m = q * per / 4; m < (q + 1) * per / 4; ++m) {
        const int i = m * kFT + tid;
        if (i < vectors) {
          uint4 v = s[i];
          clean_vector(v, top, Tag{});
          s[i] = v;
        }
      }
    }
  } else {
    F.sweep([&](int, const float (&x)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, x[j]);
    });
  }
  float hi = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  if (lane == 0) sm.part[warp][0] = hi;
  cluster_wait();                                           // every CTA of the cluster runs
  cluster_store32(cluster_map(&sm.top[F.rank * kFT + tid], 0), __float_as_uint(top));
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kFW; ++w) hi = fmaxf(hi, sm.part[w][0]);
    sm.sum[0] = Part{(double)hi, 0};
  }
  {
    const Part(*all)[kWays] = F.exchange(1);
    F.M = -INFINITY;
    for (int r = 0; r < F.G; ++r) F.M = fmaxf(F.M, (float)all[r][0].mass);
  }
  if (F.M == -INFINITY) {                                   // no token has mass
    if (F.rank == 0 && tid == 0) F.write(0, 0.0);
    return;
  }
  if (F.M == INFINITY) {                                    // the infinite ones share it
    F.M = 0.f;
    F.inf_row = true;
    if (F.resident)
      for (int i = tid; i < n; i += kFT)
        F.slice[i] = elem_of(load_generic(F.slice + i) == INFINITY ? 0.f : -INFINITY, elem{});
    if (F.rank == 0)
      for (int i = tid; i < F.G * kFT; i += kFT)
        sm.top[i] = __float_as_uint(__uint_as_float(sm.top[i]) == INFINITY ? 0.f : -INFINITY);
    __syncthreads();
  }
  if (temp == 0.f) {                                        // the argmax, lowest id
    int best = kNoIndex;
    F.sweep([&](int v, const float (&x)[8]) {
#pragma unroll
      for (int j = 7; j >= 0; --j)
        if (x[j] == F.M) best = min(best, F.id_of(v, j));
    });
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0) sm.redi[0][warp] = best;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kFW; ++w) best = min(best, sm.redi[0][w]);
      sm.sum[0] = Part{0.0, best};
    }
    const Part(*all)[kWays] = F.exchange(1);
    for (int r = 0; r < F.G; ++r) best = min(best, (int)all[r][0].count);
    if (F.rank == 0 && tid == 0) F.write(best, 1.0);
    return;
  }

  // ---- the exponent's factors; min-p as a border value
  F.Md = (double)F.M;
  F.c = 128.0 * 1.4426950408889634074 / (double)temp;
  {
    // 2^-1000 of the largest: the value nearest below it must not leave the exponent's range
    float z = fmaxf((float)(F.Md - 128000.0 / F.c), kLowest);
    while (((double)z - F.Md) * F.c < -130560.0) z = value_of(ord_of(z) + 1);
    F.zero_below = z;
  }
  float min_x = kLowest;
  if (m_on) {
    // the smallest value whose weight is min_p or more: next to its logarithm's
    unsigned o = ord_of(fmaxf((float)(F.Md + (double)temp * log((double)min_p)), kLowest));
    const unsigned om = ord_of(F.M), ol = ord_of(kLowest);
    o = min(o, om);
    o = o - ol > 4 ? o - 4 : ol;
    while (o < om && F.weight(value_of(o)) < (double)min_p) ++o;
    min_x = value_of(o) + 0.f;
  }

  // ---- what is kept
  using List = typename Filter<Tag>::List;
  unsigned long long cut = 0;
  double before;
  // a border with R tokens above it needs R maxima: of threads with a vector of their own
  const long long groups = min((long long)F.G * kFT, (long long)(a.V + W - 1) / W);
  List q{};
  q.k = 1LL << 40;
  q.P = INFINITY;
  q.top_p = 1.0;
  q.min_x = min_x;
  q.draw = true;
  bool cut_k = k_on, cut_p = p_on;
  if (a.V <= kGather || (k_on && k <= kPick)) {
    const float t = a.V <= kGather ? kLowest : F.pick((int)k);
    const int got = F.gather(t, INFINITY, 0);
    if (got <= kGather) {
      if (k_on) q.k = k;
      if (p_on) q.top_p = (double)top_p;
      F.settle(got, q, u);
      return;
    }
  } else if (p_on && !k_on) {
    const double z = F.template masses<true>(0, before), P = (double)top_p * z;
    const float t = F.pick((int)max(1LL, min((long long)kPick, groups / 4)));
    int got = F.gather(fmaxf(t, min_x), INFINITY, 0);
    float top_x = F.M;                                      // the nucleus ends below this value,
    double above = 0.0;                                     // above which lies this mass
    bool listed = false;
    if (got <= kGather) {
      q.P = P;
      q.reach = t > min_x;                                  // else all that min-p keeps is here
      if (F.settle(got, q, u)) return;
      top_x = t;
      above = sm.mass;
      listed = true;
    }
    // tokens lighter than (1 - p) z / V weigh less than (1 - p) z together: none is kept
    const double w0 = (1.0 - (double)top_p) * z / (double)a.V;
    const float x0 = (float)(F.Md + log2(w0) * 128.0 / F.c);
    float lo = fmaxf(fmaxf(x0 - fabsf(x0) * 1e-5f - 1e-30f, kLowest), min_x);
    if (!listed) top_x = value_of(ord_of(F.M) + 1);
    if (m_on && F.template masses<false>(key_floor(min_x), before) <= P) {
      cut_p = false;                                        // min-p keeps no more than top-p does
    } else if (F.narrow(lo, top_x, above, P)) {
      above = F.template masses<false>(key_floor(top_x), before);
      got = F.gather(lo, top_x, 0);
      if (got <= kGather && got > 0) {
        q.P = P;
        q.above = above;
        q.n_above = 0;
        q.min_x = kLowest;
        q.reach = true;
        q.draw = false;
        if (F.settle(got, q, u)) {
          cut = sm.cut;
          cut_p = false;
        }
      }
    }
    if (cut_p) {
      cut = F.select(0, 1LL << 40, P, true);
      cut_p = false;
    }
  } else if (m_on && !k_on) {
    // a list when few of the maxima reach the border
    const int own = F.block_count(top >= min_x, 0);
    if (tid == 0) sm.sum[0] = Part{0.0, own};
    const Part(*all)[kWays] = F.exchange(1);
    long long reach = 0;
    for (int r = 0; r < F.G; ++r) reach += all[r][0].count;
    if (reach <= min((long long)kPick, groups / 4)) {
      const int got = F.gather(min_x, INFINITY, 0);
      if (got <= kGather) {
        F.settle(got, q, u);
        return;
      }
    }
  }
  if (cut_k) cut = F.select(0, k, 0.0, false);
  if (cut_p) {
    const double z = F.template masses<false>(cut, before);
    cut = F.select(cut, 1LL << 40, (double)top_p * z, true);
  }
  if (m_on) cut = max(cut, key_floor(min_x));
  if (cut == 0) {
    const double z = F.template masses<true>(0, before);
    F.template draw<true>(0, z, before, u);
  } else {
    const double z = F.template masses<false>(cut, before);
    F.template draw<false>(cut, z, before, u);
  }
}

template <typename Tag>
cudaError_t launch_tag(FilterLaunch L, cudaStream_t stream) {
  const long long rows = (long long)L.a.B * L.a.K;
  const int chunks = (int)(((long long)L.a.V + Tag::kVec - 1 + kChunk - 1) / kChunk);   // at any alignment
  int G = kMaxCluster;
  while (G > 1 && chunks < 2 * G) G >>= 1;
  L.cluster = G;
  L.chunks_per_cta = (chunks + G - 1) / G;
  const size_t slice = (size_t)L.chunks_per_cta * kChunk * sizeof(typename Tag::elem);
  L.resident = slice <= kSliceBytes;
  const size_t smem = (sizeof(FilterSmem) + 15) / 16 * 16 + (L.resident ? slice : 0);
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
