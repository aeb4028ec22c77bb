// sample_filtered.cu -- a token per row under temperature, top-k, top-p and min-p (one launch).
//
// Every filter keeps a prefix of the order (logit descending, id ascending), so what is kept is
// "all tokens up to one cut" and the cut is a 64-bit key: the logit's order-preserving bits
// above the inverted id.  A cluster of CTAs takes a row; the first pass finds the largest logit
// and, where it will be needed, the row's mass.
//
// Two shortcuts keep those passes few.
//   A list: every thread keeps the largest logit that it loaded.  The R-th largest of these
//   maxima is a border with at least R tokens above it, and few more (tokens / threads of a row
//   are tens): the tokens above it go to one CTA, which sorts them.  With top-k (R = k) they
//   hold all that is kept; with top-p alone they do when their mass reaches p times the row's.
//   A histogram: a nucleus whose tokens are not among few maxima is closed in on by counting the
//   tokens in 4096 parts of the value range; the tokens of the part where the mass passes p make
//   the list, and the mass above them, summed in fp64, decides: the estimate is never part of an
//   answer.
// Whatever these leave open (thousands of equal logits, top_k above kPick) is narrowed exactly,
// eight ways a pass on the keys' bits (`select`).
//
// Masses are fp64 sums of fp64 exponentials: the tokens drawn are compared with an exact draw,
// and with 10^5 tokens kept every 10^-8 of error in the running mass would change one row in a
// thousand.  Sums are joined in a fixed order, so results repeat.
//
// Measured: 448 rows of 151936 fp32 logits at their temperatures: 126 us, 2.2 TB/s or 33 percent of
// the measured copy bandwidth; 35 instructions a logit, 8 of them fp64, in 60 percent of the active
// issue slots with 42 percent of the warps: latency.  768 rows of 201088 bf16 logits, each request
// with its own filters: 324 to 328 us; top-k alone 256, top-p alone 821.  7 rows: 14 to 57 us.
// The streamed kernel holds 64 registers and spills 682 (fp32) or 786 bytes, its outlined steps up to
// 1104.
#include "filter_common.cuh"
#include "kernels.h"
#include "plan.h"

namespace pspec {

namespace {

constexpr int kFT = 512;                 // threads of a CTA
constexpr int kFW = kFT / 32;
constexpr int kWays = 8;                 // parts of the bracket per pass
constexpr int kGather = 4096;            // tokens that one CTA sorts
constexpr int kPick = 1024;              // the largest rank looked for among the maxima
constexpr int kChunk = 256;              // 32 lanes x 8 elements
constexpr int kMaxCluster = 8;
constexpr long long kFewRows = 32;
constexpr int kBins = 4096;              // of a histogram
constexpr int kListV = 65536;            // (1758 rows of 4928 logits, mixed filters: 214 us, 249 with lists)
constexpr size_t kSliceBytes = 128 * 1024;   // a slice above this is read from global memory
constexpr float kLowest = -3.402823466e38f;  // tokens below it (-inf) never have mass

// The key below those of every token with this value, above all smaller ones'.
__device__ __forceinline__ unsigned long long key_floor(float x) { return (unsigned long long)ord_of(x) << 32; }

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
// No element below `least` (a pair of equal values, or an fp32 one).
__device__ __forceinline__ uint4 clamp_vector(uint4 v, uint32_t least, BF16Tag) {
  return make_uint4(max_pair(v.x, least), max_pair(v.y, least), max_pair(v.z, least), max_pair(v.w, least));
}
__device__ __forceinline__ uint4 clamp_vector(uint4 v, uint32_t least, F32Tag) {
  const float f = __uint_as_float(least);
  return make_uint4(__float_as_uint(fmaxf(__uint_as_float(v.x), f)), __float_as_uint(fmaxf(__uint_as_float(v.y), f)),
                    __float_as_uint(fmaxf(__uint_as_float(v.z), f)), __float_as_uint(fmaxf(__uint_as_float(v.w), f)));
}
__device__ __forceinline__ uint16_t elem_of(float x, uint16_t) { return (uint16_t)(__float_as_uint(x) >> 16); }
__device__ __forceinline__ float elem_of(float x, float) { return x; }
__device__ __forceinline__ float load_generic(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float load_generic(const float* p) { return *p; }

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

struct Part {            // what a CTA reports: of itself, or of one part of a bracket
  double mass;
  long long count;
};

struct FilterSmem {
  double table[128][16];                  // 2^(j/128), a copy for every lane of a half warp: random
                                          // entries of one copy would meet in the banks
  union {
    unsigned long long key[kGather];
    unsigned top[kMaxCluster * kFT];      // CTA 0: kMaxCluster / G maxima of each thread
    int bin[kBins];
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
  float pick;
  int turn;                               // the exchange buffer of the next exchange
  int ok;
  int gathered, flagged, count;
  int found, last;
};

__host__ __device__ constexpr size_t filter_smem_base() { return (sizeof(FilterSmem) + 15) / 16 * 16; }

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

template <typename Tag, bool kResident>
struct Filter {
  using elem = typename Tag::elem;
  static constexpr int W = Tag::kVec;
  static constexpr int kRaw = 8 / W;                          // 16-byte pieces of eight elements
  FilterSmem* smem;
  const double* mine;        // this lane's copy of the table
  unsigned* own;             // [parts][kFT] maxima of this CTA's threads
  uint16_t* flags;           // [parts * kFT] the ones that a gather looks behind
  int32_t* token_out;
  float* prob_out;
  const elem* row;           // the row in global memory
  elem* slice;               // this CTA's chunks in shared memory (kResident)
  int V, G, rank, tid, lane, warp;
  int lead;                  // the row is placed at this element of its first chunk, so that
                             // 16-byte aligned pieces of it are aligned in the slice too
  int c0, nc;                // this CTA's chunks [c0, c0 + nc)
  int parts;                 // maxima that a thread keeps, one for each part of its strip
  bool inf_row;              // the largest logit is +inf: those count as 0, all others as -inf
  bool far;                  // exponents beyond an integer: logits are taken relative to M
  int bias;                  // weights are in units of 2^(bias / 128), a multiple of 128
  float M, zero_below;       // largest logit; tokens below the second weigh nothing
  double c;                  // 128 log2(e) / temperature

  // exp(x / temperature) = 2^(y/128), y = x c: 2^k * table[j] * e^g with g = (y - n) ln2 / 128,
  // |g| <= 0.0028, e^g by its Taylor polynomial of degree 3 (remainder below 2.4e-12).
  // x is not below zero_below.
  template <int kMode>       // 0: bias is 0; 1: it may not be; 2: far
  __device__ __forceinline__ void factors(float x, double& scale, double& poly) const {
    constexpr bool kFar = kMode == 2;
    constexpr double a = 0.69314718055994530942 / 128.0;
    double d = (double)x;
    if (kFar) d -= (double)M;
    const double t = fma(d, c, 6755399441055744.0);          // 1.5 * 2^52: rounds to an integer
    const int n = __double2loint(t);
    const double f = fma(d, c, 6755399441055744.0 - t);
    poly = fma(f, fma(f, fma(f, a * a * a / 6.0, a * a / 2.0), a), 1.0);
    const double r = *reinterpret_cast<const double*>(reinterpret_cast<const char*>(mine) + ((n & 127) << 7));
    const int e = kMode == 1 ? (n & ~127) - bias : n & ~127;
    scale = __hiloint2double(__double2hiint(r) + (e << 13), __double2loint(r));
  }
  __device__ __forceinline__ double weight(float x) const {
    double s, p;
    const float y = fmaxf(x, zero_below);
    if (far) factors<2>(y, s, p);
    else factors<1>(y, s, p);
    return x < zero_below ? 0.0 : s * p;
  }
  // The factors before the largest logit is known: weights in units of 1, right while no logit
  // is 900 octaves away from it.
  __device__ __forceinline__ void scale_for(float temp) {
    c = 128.0 * 1.4426950408889634074 / (double)temp;
    far = false;
    bias = 0;
    zero_below = fmaxf((float)(-1020.0 * 128.0 / c), kLowest);
    while ((double)zero_below * c < -1021.0 * 128.0) zero_below = value_of(ord_of(zero_below) + 1);
  }
  // ... and whether that held; else the factors relative to it.  So hot that even the lowest finite
  // logit weighs something, -inf (clamped to it outside `far`) has to be told apart.
  __device__ __forceinline__ bool rescale() {
    const double y = (double)M * c;
    if (fabs(y) <= 900.0 * 128.0 && (double)kLowest * c <= -1020.0 * 128.0) return true;
    far = !(fabs(y) < 1073741824.0) || ((double)kLowest - (double)M) * c > -1000.0 * 128.0;
    bias = far ? 0 : 128 * (int)rint(y / 128.0);
    const double Md = (double)M;
    float z = fmaxf((float)(Md - 1000.0 * 128.0 / c), kLowest);
    while (((double)z - Md) * c < -1020.0 * 128.0) z = value_of(ord_of(z) + 1);
    zero_below = z;
    return false;
  }

  // elements 8v .. 8v + 7 of the CTA's chunks, as stored; what lies outside the row is -inf
  __device__ __forceinline__ void fetch(int v, uint4 (&raw)[kRaw]) const {
    if constexpr (kResident) {
#pragma unroll
      for (int i = 0; i < kRaw; ++i) raw[i] = *reinterpret_cast<const uint4*>(slice + (long long)v * 8 + i * W);
    } else {
#pragma unroll
      for (int i = 0; i < kRaw; ++i) {
        const int id = id_of(v, i * W);
        if (id >= 0 && id + W <= V) {
          raw[i] = ld_stream(row + id);
        } else {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            constexpr int E = W / 4;                        // elements of a word
            const float lo = inside(id + j * E), hi = E == 2 ? inside(id + j * E + 1) : 0.f;
            w[j] = E == 2 ? __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632) : __float_as_uint(lo);
          }
          raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  __device__ __forceinline__ float inside(int id) const {
    return id >= 0 && id < V ? load_scalar(row, id) : -INFINITY;
  }
  // (kClean: without NaN and -0, which comparisons do not need)
  template <bool kClean = true>
  __device__ __forceinline__ void values(const uint4 (&raw)[kRaw], float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < kRaw; ++i) {
      uint4 v = raw[i];
      if constexpr (!kResident && kClean) {                 // in shared memory they are clean
        float top = 0.f;
        clean_vector(v, top, Tag{});
      }
      float y[W];
      unpack(v, y, Tag{});
#pragma unroll
      for (int j = 0; j < W; ++j) x[i * W + j] = y[j];
    }
    if (!kResident && inf_row) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] == INFINITY ? 0.f : -INFINITY;
    }
  }
  __device__ __forceinline__ int id_of(int v, int j) const { return c0 * kChunk + v * 8 + j - lead; }

  // A warp's strip of the CTA's vectors of eight, 2 nc of them; a lane has every 32nd, and its
  // part p is the rounds [part_lo(p), part_lo(p + 1)) of them.
  __device__ __forceinline__ int strip_lo(int w) const { return nc * 2 * w; }
  __device__ __forceinline__ int rounds() const { return (nc * 2 + 31) / 32; }
  __device__ __forceinline__ int part_lo(int p) const { return rounds() * p / parts; }

  // f(v, x) for the eight elements of each of this lane's vectors, whole warps at a time; rows in
  // global memory are fetched a few vectors ahead.
  template <bool kClean = true, typename F>
  __device__ __forceinline__ void sweep(F&& f) const {
    const int lo = strip_lo(warp), hi = strip_lo(warp + 1);
    constexpr int kAhead = kResident ? 1 : 4 / kRaw;
    for (int v0 = lo; v0 < hi; v0 += 32 * kAhead) {
      uint4 raw[kAhead][kRaw];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (v0 + 32 * i + lane < hi) fetch(v0 + 32 * i + lane, raw[i]);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int v = v0 + 32 * i;
        if (i > 0 && v >= hi) break;
        float x[8];
        if (v + lane < hi) {
          values<kClean>(raw[i], x);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = -INFINITY;
        }
        f(v + lane, x);
      }
    }
  }

  // Every CTA's `n` parts sm.sum[0..n) to every CTA; all get them in rank order in the returned
  // buffer.  One cluster barrier.
  __device__ const Part (*exchange(int n))[kWays] {
    FilterSmem& sm = *smem;
    __syncthreads();
    const int turn = sm.turn;
    Part(*buf)[kWays] = sm.xch[turn];
    for (int i = tid; i < G * n; i += kFT) {
      const int to = i / n, b = i - to * n;
      const uint32_t a = cluster_map(&buf[rank][b], to);
      cluster_store(a, (unsigned long long)__double_as_longlong(sm.sum[b].mass));
      cluster_store(a + 8, (unsigned long long)sm.sum[b].count);
    }
    cluster_sync();
    if (tid == 0) sm.turn = turn ^ 1;
    return buf;
  }

  __device__ int block_count(int v, int slot) {             // alternate `slot` between calls
    FilterSmem& sm = *smem;
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
    FilterSmem& sm = *smem;
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
  template <bool kAll, int kMode>
  __device__ double masses(unsigned long long cut, double& before) {
    FilterSmem& sm = *smem;
    const float xc = kAll ? kLowest : value_of((unsigned)(cut >> 32));
    const unsigned low = (unsigned)cut;
    double a = 0.0;
    int ties = 0;                                           // of the cut's value, kept
    sweep<false>([&](int v, const float (&x)[8]) {
      const unsigned inv = 0xffffffffu - (unsigned)id_of(v, 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        double s, p;
        factors<kMode>(fmaxf(x[j], zero_below), s, p);
        // (zero_below weighs next to nothing, unless far)
        if ((kAll || x[j] > xc) && (kMode != 2 || x[j] >= zero_below)) a = fma(s, p, a);
        if (!kAll) ties += x[j] == xc && inv - j >= low;
      }
    });
    if (!kAll) a = fma((double)ties, weight(xc), a);
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
    return total(exchange(1), before);
  }
  // The mass of the tokens at or above hi, as masses() leaves it, and the ones in [lo, hi) in
  // CTA 0's keys: their number in n, above kGather when they are too many.
  template <int kMode>
  __device__ double masses_gather(float lo, float hi, int& n) {
    FilterSmem& sm = *smem;
    __syncthreads();
    if (tid == 0) sm.gathered = 0;
    __syncthreads();
    double a = 0.0;
    sweep<false>([&](int v, const float (&x)[8]) {
      unsigned in = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        double s, p;
        factors<kMode>(fmaxf(x[j], zero_below), s, p);
        if (x[j] >= hi && (kMode != 2 || x[j] >= zero_below)) a = fma(s, p, a);
        in |= x[j] >= lo && x[j] < hi ? 1u << j : 0u;
      }
      collect(v, x, in);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (lane == 0) sm.strip[warp] = a;
    __syncthreads();
    if (tid == 0) {
      double s = 0.0;
      for (int w = 0; w < kFW; ++w) s += sm.strip[w];
      sm.sum[0] = Part{s, sm.gathered};
    }
    const Part(*all)[kWays] = exchange(1);
    double before;
    const double z = total(all, before);
    n = deliver(all);
    return z;
  }
  // The list's kept tokens (sm.count of them, first in CTA 0's keys) join the strips' masses;
  // returns as masses() does.
  __device__ double join(double& before) {
    FilterSmem& sm = *smem;
    const int n = sm.count;
    if (rank > 0) {
      const uint32_t keys = cluster_map(sm.key, 0);
      for (int i = tid; i < n; i += kFT) {
        unsigned long long key;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(key) : "r"(keys + 8 * i) : "memory");
        sm.key[i] = key;
      }
    }
    __syncthreads();
    double a = 0.0;
#pragma unroll 4
    for (int i = lane; i < n; i += 32) {
      const unsigned long long key = sm.key[i];
      const int v = ((int)(0xffffffffu - (unsigned)key) + lead - c0 * kChunk) >> 3;
      if (v >= strip_lo(warp) && v < strip_lo(warp + 1)) a += weight(value_of((unsigned)(key >> 32)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (lane == 0) sm.strip[warp] += a;
    __syncthreads();
    if (tid == 0) {
      double s = 0.0;
      for (int w = 0; w < kFW; ++w) s += sm.strip[w];
      sm.sum[0] = Part{s, 0};
    }
    return total(exchange(1), before);
  }
  __device__ double total(const Part (*all)[kWays], double& before) const {
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
    FilterSmem& sm = *smem;
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
    *token_out = token;
    if (prob_out) *prob_out = (float)p;
  }

  // ------------------------------------------------------------------ the list
  // The border: a value with at least R of the maxima, and few more, at or above it (kLowest
  // when fewer are finite); with a mass P, one with as few of them as weigh P (sm.ok: there is).
  // CTA 0 looks, all get the answer.  The first cluster barrier of the row must lie between the
  // maxima's stores and this.
  __device__ float pick(int R, double P) {
    FilterSmem& sm = *smem;
    if (rank == 0) {
      constexpr int kPer = kMaxCluster;
      float x[kPer], w[kPer];
      float least = INFINITY, sum = 0.f;
      int finite = 0;
      const float cf = (float)(c / 128.0), limit = (float)(P * (1.0 + 1e-5));
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        x[i] = __uint_as_float(sm.top[i * kFT + tid]);
        w[i] = 0.f;
        if (x[i] > -INFINITY) {
          least = fminf(least, x[i]);
          ++finite;
          w[i] = ex2((x[i] - M) * cf);
        }
        sum += w[i];
      }
      const bool by_mass = block_mass(sum, 0) >= limit;     // false for P = INFINITY
      // the smallest finite maximum, as an integer of the same order
      const unsigned o = __reduce_min_sync(0xffffffffu, ord_of(least));
      if (lane == 0) sm.redi[0][warp] = (int)o;
      __syncthreads();
      unsigned lo_o = 0xffffffffu;
      for (int w = 0; w < kFW; ++w) lo_o = min(lo_o, (unsigned)sm.redi[0][w]);
      float t = kLowest;
      const bool enough = block_count(finite, 1) >= R;
      if (enough || by_mass) {
        float lo = value_of(lo_o), hi = M;                  // the maxima at or above lo are enough
        t = lo;
        for (int step = 0; step < 24; ++step) {
          const float mid = 0.5f * lo + 0.5f * hi;
          if (!(mid > lo)) break;
          int n = 0;
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            n += x[i] >= mid;
            s += x[i] >= mid ? w[i] : 0.f;
          }
          n = block_count(n, step & 1);
          const bool heavy = by_mass && block_mass(s, step & 1) >= limit;
          if (by_mass ? heavy : n >= R) {
            t = lo = mid;
            if (n <= (by_mass ? kFT / 4 : R + R / 8 + 4)) break;
          } else {
            if (mid == hi) break;
            hi = mid;
          }
        }
      }
      if (tid < G) {
        cluster_store32(cluster_map(&sm.pick, tid), __float_as_uint(t));
        cluster_store32(cluster_map(&sm.ok, tid), by_mass);
      }
    }
    cluster_sync();
    return sm.pick;
  }
  __device__ float block_mass(float v, int slot) {          // alternate `slot` between calls
    FilterSmem& sm = *smem;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) sm.part[warp][slot] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kFW; ++w) s += sm.part[w][slot];
    return s;
  }

  // The tokens with lo <= x < hi and key >= cut (hi: +inf for no limit; lo is not below the cut's
  // value) into CTA 0's keys, in no fixed order; returns how many, and copies nothing when they
  // are more than kGather.  Two cluster barriers.
  __device__ int gather(float lo, float hi, unsigned long long cut) {
    FilterSmem& sm = *smem;
    const unsigned low = value_of((unsigned)(cut >> 32)) == lo ? (unsigned)cut : 0u;
    __syncthreads();
    if (tid == 0) sm.gathered = sm.flagged = 0;
    __syncthreads();
    for (int p = 0; p < parts; ++p) {
      const bool in = __uint_as_float(own[p * kFT + tid]) >= lo;
      const unsigned all = __ballot_sync(0xffffffffu, in);
      int at = 0;
      if (lane == 0 && all) at = atomicAdd(&sm.flagged, __popc(all));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(all & ((1u << lane) - 1u));
      if (in) flags[at] = (uint16_t)(p * kFT + tid);
    }
    __syncthreads();
    // a part's pieces go to as many threads; the last parts may be a round shorter
    const int nf = sm.flagged, most = (rounds() + parts - 1) / parts;
    for (int i0 = 0; i0 < nf * most; i0 += kFT) {
      const int i = i0 + tid;
      float x[8];
      int v = 0;
      bool there = i < nf * most;
      if (there) {
        const int m = i / nf, e = flags[i - m * nf], p = e / kFT, t = e - p * kFT;
        const int round = part_lo(p) + m;
        v = strip_lo(t >> 5) + round * 32 + (t & 31);
        there = round < part_lo(p + 1) && v < strip_lo((t >> 5) + 1);
      }
      if (there) {
        uint4 raw[kRaw];
        fetch(v, raw);
        values(raw, x);
      }
      unsigned in = 0;
      if (there) {
#pragma unroll
        for (int j = 0; j < 8; ++j) in |= (x[j] >= lo && x[j] < hi ? 1u : 0u) << j;
        if (low != 0) {                                     // a cut inside the ties of its value
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (x[j] == lo && 0xffffffffu - (unsigned)id_of(v, j) < low) in &= ~(1u << j);
        }
      }
      collect(v, x, in);
    }
    __syncthreads();
    if (tid == 0) sm.sum[0] = Part{0.0, sm.gathered};
    return deliver(exchange(1));
  }
  // The elements of x named by the bits of `in` into this CTA's keys.
  __device__ __forceinline__ void collect(int v, const float (&x)[8], unsigned in) const {
    if (in == 0) return;
    int at = atomicAdd(&smem->gathered, __popc(in));
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (in >> j & 1) {
        if (at < kGather) smem->key[at] = key_of(x[j] + 0.f, id_of(v, j));
        ++at;
      }
  }
  // Every CTA's keys, counted in `all`, to CTA 0.  One cluster barrier.
  __device__ int deliver(const Part (*all)[kWays]) {
    FilterSmem& sm = *smem;
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
  // With `reach` or without `draw`, whether the list held the cut, the cut and the number of tokens up
  // to it go to every CTA's sm.ok, sm.cut and sm.count, and the cluster barrier is arrived at.
  template <int kPer>
  __device__ void settle(int n, List q, double u) {
    FilterSmem& sm = *smem;
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
      if (!q.draw) {                                        // the list in order, for join()
#pragma unroll
        for (int r = 0; r < kPer; ++r) sm.key[tid * kPer + r] = key[r];
      }
#pragma unroll
      for (int r = 0; r < kPer; ++r)
        if (tid * kPer + r == m - 1)
          for (int g = 0; g < G; ++g) cluster_store(cluster_map(&sm.cut, g), key[r]);
      if (tid < G) {
        cluster_store32(cluster_map(&sm.ok, tid), ok);
        cluster_store32(cluster_map(&sm.count, tid), m);
      }
      cluster_arrive();
    }
    if (!ok || !q.draw) return;
    // the kept tokens in id order: sorted by the inverted id, which is the keys' low half
#pragma unroll
    for (int r = 0; r < kPer; ++r)
      key[r] = tid * kPer + r < m ? key[r] << 32 | key[r] >> 32 : 0;
    if (kPer > 1 && m <= kFT) {
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kPer; ++r)
        if (tid * kPer + r < kFT) sm.key[tid * kPer + r] = key[r];
      __syncthreads();
      unsigned long long one[1] = {sm.key[tid]};
      draw_list<1>(one, m, u);
    } else {
      draw_list<kPer>(key, m, u);
    }
  }
  // The draw among the m keys (inverted id, logit), zeros behind them.
  template <int kPer>
  __device__ void draw_list(unsigned long long (&key)[kPer], int m, double u) {
    FilterSmem& sm = *smem;
    sort<kPer>(key);
    double w[kPer], s = 0.0, all;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      w[r] = tid * kPer + r < m ? weight(value_of((unsigned)key[r])) : 0.0;
      s += w[r];
    }
    if (tid == 0) {
      sm.found = kNoIndex;
      sm.last = -1;
    }
    double at = block_scan(s, all);
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
    FilterSmem& sm = *smem;
    const bool answer = q.reach || !q.draw;
    if (rank == 0) {
      if (n <= kFT) settle<1>(n, q, u);
      else if (n <= 4 * kFT) settle<4>(n, q, u);
      else settle<kGather / kFT>(n, q, u);
    } else if (answer) {
      cluster_arrive();
    }
    if (!answer) return true;
    cluster_wait();
    return sm.ok != 0;
  }

  // ------------------------------------------------------------------ the histogram
  // Closes [lo, hi) in on the value at which the mass above passes P, given the mass A above hi
  // (both in units of the largest weight): tokens are counted in kBins equal parts, and a part's
  // mass lies within e^(+-half its width) of its count times its middle's weight.  Returns the
  // tokens counted in the new bracket, those above it up to the old one in n_above; 0: the mass
  // stays below P; -1: no answer.
  __device__ int histogram(float& lo_out, float& hi_out, double A, double P, int& n_above) {
    FilterSmem& sm = *smem;
    const float lo = lo_out, hi = hi_out;
    const float span = hi - lo, s = (float)(kBins - 1) / span, cf = (float)(c / 128.0);
    if (!(span > 0.f) || !(s < 1e30f) || !(s > 0.f)) return -1;
    const uint32_t bins = (uint32_t)__cvta_generic_to_shared(sm.bin);
    __syncthreads();
    for (int i = tid; i < kBins; i += kFT) sm.bin[i] = 0;
    __syncthreads();
    sweep<false>([&](int, const float (&x)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // the nearest of the parts' middles, as the low bits of a float above 2^23
        const float at = fmaf(x[j] - lo, s, 8388608.f);
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ge.f32 p, %0, %1;\n\tsetp.lt.and.f32 q, %0, %2, p;\n\t"
                     "@q red.shared.add.u32 [%3], 1;\n\t}" ::"f"(x[j]), "f"(lo), "f"(hi),
                     "r"(bins + ((__float_as_uint(at) & (2 * kBins - 1)) << 2)));      // (read behind the cluster barrier)
      }
    });
    cluster_sync();
    constexpr int kPer = kBins / kFT;
    int count[kPer];
    double mass = 0.0, cum[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {                        // thread 0 has the highest part
      const int b = kBins - 1 - (tid * kPer + i);
      count[i] = 0;
      for (int r = 0; r < G; ++r) {
        int n;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(n) : "r"(cluster_map(&sm.bin[b], r)) : "memory");
        count[i] += n;
      }
      mass += (double)count[i] * (double)ex2((lo + (float)b / s - M) * cf);
      cum[i] = mass;
    }
    double all;
    const double base = block_scan(mass, all);
    const double slack = (double)ex2(0.5f * cf / s) * (1.0 + 1e-5);
    int sure = 0, reach = 0;                                // parts whose mass up to them is below P for
#pragma unroll                                              // sure; that need not reach P
    for (int i = 0; i < kPer; ++i) {
      const double m = base + cum[i];
      sure += A + m * slack < P;
      reach += A + m / slack < P;
    }
    __syncthreads();
    sure = block_count(sure, 0);
    reach = block_count(reach, 1);
    __syncthreads();
    const int from = max(0, sure - 1), to = min(kBins, reach + 2);     // a part more on each side
    int in = 0, above = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * kPer + i;
      above += b < from ? count[i] : 0;
      in += b >= from && b < to ? count[i] : 0;
    }
    in = block_count(in, 0);
    n_above = block_count(above, 1);
    cluster_sync();                                         // the others have read the parts
    if (sure >= kBins) return 0;
    if (from > 0) hi_out = lo + ((float)(kBins - from) - 0.5f) / s;
    if (to < kBins) lo_out = lo + ((float)(kBins - to) - 0.5f) / s;
    return in > 0 ? in : -1;                                // (estimates that are not finite say nothing)
  }

  // ------------------------------------------------------------------ exact narrowing
  // The cut under "rank < k" and "mass before < P" among the tokens with key >= old.
  // `need_mass`: P is a limit.
  __device__ unsigned long long select(unsigned long long old, long long k, double P, bool need_mass) {
    FilterSmem& sm = *smem;
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
    FilterSmem& sm = *smem;
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
    FilterSmem& sm = *smem;
    // which CTA: the first whose running mass passes u z, else the last with mass
    __syncthreads();
    const Part(*all)[kWays] = sm.xch[sm.turn ^ 1];          // the last exchange: the masses
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
    // which of the strip's rounds: every warp sums a run of them
    const int at_strip = strip >= 0 ? strip : end;
    const int v_lo = strip_lo(at_strip), v_hi = strip_lo(at_strip + 1), n = rounds();
    const float xc = kAll ? kLowest : value_of((unsigned)(cut >> 32));
    const unsigned low = (unsigned)cut;
    auto kept = [&](int v, float x, int j) {
      return kAll || x > xc || (x == xc && 0xffffffffu - (unsigned)id_of(v, j) >= low) ? weight(x) : 0.0;
    };
    auto load = [&](int round, float (&x)[8]) {
      const int v = v_lo + round * 32 + lane;
      if (v < v_hi) {
        uint4 raw[kRaw];
        fetch(v, raw);
        values(raw, x);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = -INFINITY;
      }
      return v;
    };
    double sum = 0.0;
    for (int r = n * warp / kFW; r < n * (warp + 1) / kFW; ++r) {
      float x[8];
      const int v = load(r, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += kept(v, x[j], j);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sm.red[warp] = sum;
    __syncthreads();
    if (warp != 0) return;
    int run_at = -1;
    end = 0;
    base = start;
    for (int i = 0; i < kFW; ++i) {
      const double t = sm.red[i];
      if (t > 0.0) {
        if (run_at < 0) start = base;
        end = i;
        if (run_at < 0 && strip >= 0 && base + t > thr) run_at = i;
      }
      base += t;
    }
    const int at_run = run_at >= 0 ? run_at : end;
    // which token: the run's rounds in turn
    double run = run_at >= 0 ? start : -INFINITY;
    int first = kNoIndex, tail = -1;
    double wf = 0.0, wt = 0.0;
    for (int round = n * at_run / kFW; round < n * (at_run + 1) / kFW && first == kNoIndex; ++round) {
      float x[8];
      const int v = load(round, x);
      double w[8], s = 0.0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = kept(v, x[j], j);
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
    }
    if (first != kNoIndex) {
      if (wf > 0.0) write(first, wf / z);
    } else if (wt > 0.0) {
      write(tail, wt / z);
    }
  }
};

// The row of a batch that cluster `at` takes when the sequences under top-p alone, whose nuclei may
// take several passes, come first (else they end last, alone: 768 rows under mixed filters 327 us, 460 in order).
__device__ __forceinline__ long long heavy_first_row(const pspec_filter_args& a, FilterSmem& sm, long long at) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int j = (int)(at / a.K);
  auto heavy = [&](int i) {
    return __ldg(a.top_p + i) < 1.f && !(a.top_k && __ldg(a.top_k + i) > 0) && !(a.temperature && __ldg(a.temperature + i) == 0.f);
  };
  int n = 0;
  for (int i = tid; i < a.B; i += kFT) n += heavy(i);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) sm.redi[0][warp] = n;
  __syncthreads();
  n = 0;
  for (int w = 0; w < kFW; ++w) n += sm.redi[0][w];
  const bool side = j < n;
  int want = side ? j : j - n;
  for (int base = 0; base < a.B; base += kFT) {             // the want-th sequence of its side
    const bool in = base + tid < a.B && heavy(min(base + tid, a.B - 1)) == side;
    const unsigned all = __ballot_sync(0xffffffffu, in);
    __syncthreads();
    if (lane == 0) sm.redi[1][warp] = __popc(all);
    __syncthreads();
    int before = __popc(all & ((1u << lane) - 1u)), total = 0;
    for (int w = 0; w < kFW; ++w) {
      before += w < warp ? sm.redi[1][w] : 0;
      total += sm.redi[1][w];
    }
    if (in && before == want) sm.found = base + tid;
    want -= total;
    if (want < 0) break;
  }
  __syncthreads();
  return (long long)sm.found * a.K + (at - (long long)j * a.K);
}

// The rarer or larger steps once in the code each, on a copy of the state: its members stay in
// the kernel's registers.
template <typename F>
__device__ __noinline__ float call_pick(F x, int R, double P) {
  F f = x;
  return f.pick(R, P);
}
template <typename F>
__device__ __noinline__ int call_gather(F x, float lo, float hi, unsigned long long cut) {
  F f = x;
  return f.gather(lo, hi, cut);
}
template <typename F>
__device__ __noinline__ bool call_settle(F x, int n, typename F::List q, double u) {
  F f = x;
  return f.settle(n, q, u);
}
template <typename F>
__device__ __noinline__ int call_histogram(F x, float& lo, float& hi, double A, double P, int& n_above) {
  F f = x;
  return f.histogram(lo, hi, A, P, n_above);
}
template <typename F>
__device__ __noinline__ unsigned long long call_select(F x, unsigned long long old, long long k, double P, bool need_mass) {
  F f = x;
  return f.select(old, k, P, need_mass);
}
template <typename F>
__device__ __noinline__ double call_masses_gather(F x, float lo, float hi, int& n) {
  F f = x;
  return f.far ? f.template masses_gather<2>(lo, hi, n) : f.template masses_gather<1>(lo, hi, n);
}
template <typename F>
__device__ __noinline__ double call_masses(F x, unsigned long long cut, double& before) {
  F f = x;
  if (f.far) return f.template masses<false, 2>(max(cut, key_floor(kLowest)), before);
  return cut == 0 ? f.template masses<true, 1>(0, before) : f.template masses<false, 1>(cut, before);
}

template <typename Tag, bool kResident>
__global__ void __launch_bounds__(kFT, 2) filter_kernel(const FilterLaunch L) {
  using elem = typename Tag::elem;
  using Fn = Filter<Tag, kResident>;
  constexpr int W = Tag::kVec, kRaw = Fn::kRaw;
  extern __shared__ __align__(16) uint8_t s_raw[];
  FilterSmem& sm = *reinterpret_cast<FilterSmem*>(s_raw);
  const pspec_filter_args& a = L.a;
  cluster_arrive();                                         // waited for before the first remote store
  Fn F;
  F.smem = &sm;
  F.mine = &sm.table[0][threadIdx.x & 15];
  F.V = a.V;
  F.G = L.cluster;
  F.rank = cluster_rank();
  F.tid = threadIdx.x;
  F.lane = threadIdx.x & 31;
  F.warp = threadIdx.x >> 5;
  const int tid = F.tid, lane = F.lane, warp = F.warp;
  long long at = blockIdx.x / L.cluster;
  if (!kResident && L.heavy_first) at = heavy_first_row(a, sm, at);
  const long long seq = at / a.K;
  F.row = static_cast<const elem*>(a.logits) + at * a.ld;
  F.token_out = a.tokens + at;
  F.prob_out = a.probs ? a.probs + at : nullptr;
  F.lead = (int)((reinterpret_cast<uintptr_t>(F.row) & 15u) / sizeof(elem));
  const int chunks = (int)(((long long)a.V + F.lead + kChunk - 1) / kChunk);
  F.c0 = min(chunks, F.rank * L.chunks_per_cta);
  F.nc = min(chunks - F.c0, L.chunks_per_cta);
  F.parts = kMaxCluster / F.G;
  F.own = reinterpret_cast<unsigned*>(s_raw + filter_smem_base());
  F.flags = reinterpret_cast<uint16_t*>(F.own + F.parts * kFT);
  F.slice = reinterpret_cast<elem*>(F.flags + F.parts * kFT);
  F.inf_row = false;
  const int v_lo = F.strip_lo(warp), v_hi = F.strip_lo(warp + 1), rounds = F.rounds();

  // ---- the slice into shared memory: every lane the pieces that it sweeps, in flight together;
  // pieces at the row's ends by elements
  if constexpr (kResident) {
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(F.slice);
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      for (int m = q * rounds / 4; m < (q + 1) * rounds / 4; ++m) {
        const int v = v_lo + m * 32 + lane;
        if (v >= v_hi) break;
#pragma unroll
        for (int r = 0; r < kRaw; ++r) {
          const int id = F.id_of(v, r * W), i = v * 8 + r * W;
          if (id >= 0 && id + W <= a.V) {
            copy16(dst + i * (int)sizeof(elem), F.row + id);
          } else {
            for (int j = 0; j < W; ++j) F.slice[i + j] = elem_of(F.inside(id + j), elem{});
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }

  // ---- parameters
  if (tid < 128) {
    const double e = exp2((double)tid / 128.0);
    for (int i = 0; i < 16; ++i) sm.table[tid][(i + tid) & 15] = e;
  }
  if (tid == 0) sm.turn = 0;
  const FilterParams prm = filter_params(a, seq, F.rank == 0 && tid == 0);
  const float temp = prm.temperature, top_p = prm.top_p, min_p = prm.min_p;
  const long long k = prm.k;
  const double u = (double)__ldg(a.uniforms + at);
  const bool k_on = prm.k_on, p_on = prm.p_on, m_on = prm.m_on;
  // a list needs no mass of the row, and most min-p sets make one
  const bool list_k = k_on && k <= kPick;
  const bool mass_first = temp > 0.f && !list_k && !(m_on && !p_on);
  F.scale_for(temp);
  F.M = 0.f;
  __syncthreads();

  // ---- the first pass: NaN and -0 taken out, each part's largest logit, the row's mass
  float hi = -INFINITY;
  double mass = 0.0;
  // (negative, so that dropping bits rounds up)
  const unsigned floor_bits = __float_as_uint(F.zero_below);
  const uint32_t floor_pair = W == 8 ? __byte_perm(floor_bits, 0, 0x3232) : floor_bits;
  auto pass = [&](auto with_mass) {
    constexpr int kAhead = kResident ? 1 : 4 / kRaw;
    for (int p = 0; p < F.parts; ++p) {
      const int end = F.part_lo(p + 1);
      float top = -INFINITY;
      for (int m0 = F.part_lo(p); m0 < end; m0 += kAhead) {
        uint4 raw[kAhead][kRaw];
        if constexpr (kResident) {
          // the groups of copies end at q rounds / 4
          if (m0 == 0) asm volatile("cp.async.wait_group 3;" ::: "memory");
          if (m0 == rounds / 4) asm volatile("cp.async.wait_group 2;" ::: "memory");
          if (m0 == 2 * rounds / 4) asm volatile("cp.async.wait_group 1;" ::: "memory");
          if (m0 == 3 * rounds / 4) asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int v = v_lo + (m0 + i) * 32 + lane;
          if (m0 + i < end && v < v_hi) F.fetch(v, raw[i]);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int v = v_lo + (m0 + i) * 32 + lane;
          if (m0 + i < end && v < v_hi) {
#pragma unroll
            for (int r = 0; r < kRaw; ++r) {
              clean_vector(raw[i][r], top, Tag{});
              if constexpr (kResident) *reinterpret_cast<uint4*>(F.slice + v * 8 + r * W) = raw[i][r];
            }
            if constexpr (decltype(with_mass)::value) {
#pragma unroll
              for (int r = 0; r < kRaw; ++r) {
                float x[W];
                unpack(clamp_vector(raw[i][r], floor_pair, Tag{}), x, Tag{});
#pragma unroll
                for (int j = 0; j < W; ++j) {
                  double s, q;
                  F.template factors<0>(x[j], s, q);
                  mass = fma(s, q, mass);
                }
              }
            }
          }
        }
      }
      F.own[p * kFT + tid] = __float_as_uint(top);
      hi = fmaxf(hi, top);
    }
  };
  if (mass_first) pass(Yes{});
  else pass(No{});
  float largest = hi;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, o));
    mass += __shfl_xor_sync(0xffffffffu, mass, o);
  }
  if (lane == 0) {
    sm.part[warp][0] = largest;
    sm.strip[warp] = mass;
  }
  cluster_wait();                                           // every CTA of the cluster runs
  for (int p = 0; p < F.parts; ++p)
    cluster_store32(cluster_map(&sm.top[(F.rank * F.parts + p) * kFT + tid], 0), F.own[p * kFT + tid]);
  __syncthreads();
  if (tid == 0) {
    mass = sm.strip[0];
    for (int w = 1; w < kFW; ++w) {
      largest = fmaxf(largest, sm.part[w][0]);
      mass += sm.strip[w];
    }
    sm.sum[0] = Part{mass, (long long)__float_as_int(largest)};
  }
  double z, before;
  {
    const Part(*all)[kWays] = F.exchange(1);
    F.M = -INFINITY;
    for (int r = 0; r < F.G; ++r) F.M = fmaxf(F.M, __int_as_float((int)all[r][0].count));
    z = F.total(all, before);
  }
  if (F.M == -INFINITY) {                                   // no token has mass
    if (F.rank == 0 && tid == 0) F.write(0, 0.0);
    return;
  }
  bool have_mass = mass_first;
  if (F.M == INFINITY) {                                    // the infinite ones share it
    F.M = 0.f;
    F.inf_row = true;
    have_mass = false;
    auto swap = [](float x) { return x == INFINITY ? 0.f : -INFINITY; };
    if (kResident)
      for (int i = tid; i < F.nc * kChunk; i += kFT) F.slice[i] = elem_of(swap(load_generic(F.slice + i)), elem{});
    for (int i = tid; i < F.parts * kFT; i += kFT) F.own[i] = __float_as_uint(swap(__uint_as_float(F.own[i])));
    if (F.rank == 0)
      for (int i = tid; i < kMaxCluster * kFT; i += kFT) sm.top[i] = __float_as_uint(swap(__uint_as_float(sm.top[i])));
    hi = swap(hi);
    __syncthreads();
  }
  if (temp == 0.f) {                                        // the argmax, lowest id
    int best = kNoIndex;
    if (__any_sync(0xffffffffu, hi == F.M))
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
  if (!F.rescale()) have_mass = false;

  // ---- min-p as a border value: the smallest whose weight is min_p of the largest, or more
  float min_x = kLowest;
  if (m_on) {
    unsigned o = ord_of(fmaxf((float)((double)F.M + (double)temp * log((double)min_p)), kLowest));
    const unsigned om = ord_of(F.M), ol = ord_of(kLowest);
    const double limit = (double)min_p * F.weight(F.M);
    o = min(o, om);
    o = o - ol > 4 ? o - 4 : ol;
    // The border lies a few values above o, as a rule.  Near 0, and at high temperatures, values lie closer
    // than weights are resolved (2.4e-12), and it may be a billion of them away, on either side.
    auto holds = [&](unsigned at) { return F.weight(value_of(at)) >= limit; };      // true of om
    unsigned lo = o, hi = om;
    if (holds(lo)) {
      hi = lo;
      lo = ol;
      if (holds(lo)) hi = lo;
    } else {
      for (int i = 0; i < 8 && hi > lo + 1; ++i) {
        if (holds(lo + 1)) hi = lo + 1;
        else ++lo;
      }
    }
    while (hi > lo + 1) {                                   // lo does not hold, hi does
      const unsigned mid = lo + (hi - lo) / 2;
      if (holds(mid)) hi = mid;
      else lo = mid;
    }
    min_x = value_of(hi) + 0.f;
  }

  // ---- what is kept
  unsigned long long cut = 0;
  // as many maxima as there are threads' parts, and pieces of a row
  const long long groups = min((long long)kMaxCluster * kFT, (long long)(a.V + 7) / 8);
  typename Fn::List q{};
  q.k = 1LL << 40;
  q.P = INFINITY;
  q.top_p = 1.0;
  q.min_x = min_x;
  q.draw = true;
  bool cut_k = k_on, cut_p = p_on;
  if (list_k) {
    const float t = call_pick(F, (int)k, (double)INFINITY);
    const int got = call_gather(F, t, INFINITY, 0);
    if (got <= kGather) {
      q.k = k;
      if (p_on) q.top_p = (double)top_p;
      call_settle(F, got, q, u);
      return;
    }
  } else if (p_on && !k_on) {
    if (!have_mass) z = call_masses(F, 0, before);
    const double P = (double)top_p * z, unit = F.weight(F.M);
    const float t = call_pick(F, kNoIndex, P / unit);
    int got = kGather + 1;
    q.P = P;
    if (sm.ok) {                                            // few maxima hold the nucleus
      got = call_gather(F, fmaxf(t, min_x), INFINITY, 0);
      q.reach = t > min_x;                                  // else all that min-p keeps is here
      if (got <= kGather && call_settle(F, got, q, u)) return;
    }
    // tokens lighter than (1 - p) z / V weigh less than (1 - p) z together: none is kept
    const double w0 = (1.0 - (double)top_p) * (z / unit) / (double)a.V;
    const float x0 = (float)((double)F.M + log2(w0) * 128.0 / F.c);
    float lo = fmaxf(fmaxf(x0 - fabsf(x0) * 1e-5f - 1e-30f, kLowest), min_x);
    float top_x = value_of(ord_of(F.M) + 1);                // the nucleus ends below this value,
    double above = 0.0;                                     // above which lies this mass
    for (int tries = 0; tries < 3 && cut_p; ++tries) {
      int n_above;
      const int in = call_histogram(F, lo, top_x, above / unit, P / unit, n_above);
      if (in == 0 && m_on && tries == 0) {                  // min-p keeps no more than top-p does
        cut_p = false;
        break;
      }
      if (in <= 0) break;
      q.reach = true;
      // all that is kept makes a list after all: a short one, or one that sorts sooner than the
      // row's masses are summed
      if (tries == 0 && (n_above + in <= kFT || (n_above + in <= kGather && a.V > kListV))) {
        got = call_gather(F, lo, INFINITY, 0);
        if (got <= kGather && call_settle(F, got, q, u)) return;
        break;
      }
      above = call_masses_gather(F, lo, top_x, got);
      if (got > kGather) continue;
      if (got <= 0) break;
      q.above = above;
      q.min_x = kLowest;
      q.draw = false;
      if (call_settle(F, got, q, u)) {
        cut = sm.cut;
        cut_p = false;
        if (!m_on || cut >= key_floor(min_x)) {
          z = F.join(before);
          F.template draw<false>(cut, z, before, u);
          return;
        }
      }
      break;
    }
    if (cut_p && m_on && call_masses(F, key_floor(min_x), before) <= P) cut_p = false;
    if (cut_p) cut = call_select(F, 0, 1LL << 40, P, true);
    cut_p = false;
    have_mass = false;
  } else if (m_on && !k_on) {
    // a list when few of the maxima reach the border
    int own = 0;
    for (int i = tid; i < F.parts * kFT; i += kFT) own += __uint_as_float(F.own[i]) >= min_x;
    own = F.block_count(own, 0);
    if (tid == 0) sm.sum[0] = Part{0.0, own};
    const Part(*all)[kWays] = F.exchange(1);
    long long reach = 0;
    for (int r = 0; r < F.G; ++r) reach += all[r][0].count;
    if (reach <= min((long long)kPick, groups / 4)) {
      const int got = call_gather(F, min_x, INFINITY, 0);
      if (got <= kGather) {
        call_settle(F, got, q, u);
        return;
      }
    }
  }
  if (cut_k) cut = call_select(F, 0, k, 0.0, false);
  if (cut_p) {
    z = call_masses(F, cut, before);
    cut = call_select(F, cut, 1LL << 40, (double)top_p * z, true);
  }
  if (m_on) cut = max(cut, key_floor(min_x));
  if (cut != 0 || !have_mass) z = call_masses(F, cut, before);
  if (cut == 0) F.template draw<true>(0, z, before, u);
  else F.template draw<false>(cut, z, before, u);
}

template <typename Tag, bool kResident>
cudaError_t launch_kind(const FilterLaunch& L, size_t smem, cudaStream_t stream) {
  auto* fn = filter_kernel<Tag, kResident>;
  // The limit belongs to the function, not to this call: always the largest that any call takes, so
  // that no other host thread's launch finds it lowered.
  constexpr size_t most = filter_smem_base() + (size_t)kMaxCluster * kFT * 6 + (kResident ? kSliceBytes : 0);
  static_assert(most <= 227 * 1024, "within the SM's");
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = L.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((long long)L.a.B * L.a.K * L.cluster));
  cfg.blockDim = dim3(kFT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fn, L);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename Tag>
cudaError_t launch_tag(FilterLaunch L, cudaStream_t stream) {
  const long long rows = (long long)L.a.B * L.a.K;
  const int chunks = (int)(((long long)L.a.V + Tag::kVec - 1 + kChunk - 1) / kChunk);   // at any alignment
  // Few rows: the most CTAs a row, its slices in shared memory (7 rows of 201088 bf16 logits: 21 us
  // against 42 by one CTA a row; 64 rows of 5000, 69 us by two with slices, 79 without, so the border
  // could lie higher).  Many: fewer CTAs a row, which meet less, and read it again from L2, where
  // more loads are in flight than a slice in shared memory leaves room for.
  const bool few = rows <= kFewRows;
  int G = kMaxCluster;
  // With many rows, G CTAs to one take G times the waves (of two CTAs an SM), each with its meetings,
  // which are worth some 48 chunks of a CTA's part; the last rows end sooner by their longer parts.  Of
  // 13 batches of 33 to 2000 rows x 8 vocabularies of 2300 to 201088 bf16 logits this takes 1.3 percent
  // longer than the best G under mixed filters, 4 under any one (a fixed number of CTAs: 3 and 8).  E.g.
  // mixed, us by one, two and four CTAs: 769 rows of 151936 427, 324, 497; 768 of 40000 157, 221, 368;
  // 200 of 201088 353, 230, 204.
  // (A CTA's part of a row is not so short that meeting takes longer: 248 rows of 2371 tokens, top-p,
  // 62 us by one CTA, 246 by four.)
  while (G > 1 && (chunks < (few ? 16 : 64) * G || (!few && rows * G * G * 48 > 2LL * kNumSMs * chunks))) G >>= 1;
  L.cluster = G;
  L.chunks_per_cta = (chunks + G - 1) / G;
  const size_t slice = (size_t)L.chunks_per_cta * kChunk * sizeof(typename Tag::elem);
  const size_t base = filter_smem_base() + (size_t)(kMaxCluster / G) * kFT * 6;
  if (few && slice <= kSliceBytes) return launch_kind<Tag, true>(L, base + slice, stream);
  // (every CTA looks the sequences over: not for thousands of them)
  L.heavy_first = L.a.top_p && L.a.B > 1 && L.a.B <= 4096 && rows * G > 2 * kNumSMs;
  return launch_kind<Tag, false>(L, base, stream);
}

}  // namespace

cudaError_t launch_filter(const FilterLaunch& L, cudaStream_t stream) {
  if (L.a.V <= kFilterSmallV) return launch_filter_small(L, stream);
  return L.a.dtype == PSPEC_BF16 ? launch_tag<BF16Tag>(L, stream) : launch_tag<F32Tag>(L, stream);
}

}  // namespace pspec
