// append_kv.cu -- keys and values into the paged cache, rotated to their positions (one
// launch), with the query rows rotated beside them.
//
// A row goes to a CTA, or to a warp when there are many: every thread owns the same eight
// elements of each head that it comes to, and fetches a few heads ahead.
// Partners of the half split come from the lane that holds them where a head's lanes lie in one
// warp.  The first heads are on their way while the sines and cosines of the row's angles are
// formed, once for all heads.  Angles pos * inv_freq are formed and reduced in fp64 (positions
// reach 10^6: an fp32 product would be off by 0.06 rad there), rotations run in fp32.
//
// 4-bit cache: two lanes share a block of 16 elements.  Which code a value takes is decided as
// if computed exactly, and fp32 decides nearly always: the scale and the codes are rounded at
// both ends of the interval that holds the exact value, and where the ends differ (a few blocks
// in ten thousand) the block is done again in fp64, whose borders mid * s * g (3 + 4 + 24
// significant bits) are exact, so that ties are seen as ties.
//
// Measured: 15360 rows (a quarter of them padding) of 64 query and 2 x 8 key and value heads of 64
// bf16, to 4 bits with the stored values written out: 68 us, 3.6 TB/s or 55 percent of the measured
// copy bandwidth.  Neither bytes nor instructions fill it (64 percent of the active issue slots, half
// of the integer pipe): 72 registers leave room for 31 percent of the warps, which wait for loads and
// for one another's results.  A call for 15 rows takes 8 to 9 us from the host, which is its launch (a
// call of padding rows alone takes as long); inside a graph 6.4 us, 1.1 with padding alone: one row's
// chain of loads, angles and stores.  The 4-bit kernels spill up to 52 bytes, the fp64 step at most.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "plan.h"

namespace pspec {

namespace {

template <typename Tag> struct Row;
template <> struct Row<BF16Tag> {
  static constexpr int kRaw = 1, kAhead = 4;    // 16-byte pieces of eight elements; heads in flight
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ void store8(uint16_t* p, bool vec, const float (&x)[8]) {
    const uint4 v = make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7]));
    if (vec) {
      *reinterpret_cast<uint4*>(p) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
  }
};
template <> struct Row<F32Tag> {
  static constexpr int kRaw = 2, kAhead = 2;
  static __device__ __forceinline__ uint32_t pack(float lo, float) { return __float_as_uint(lo); }
  static __device__ __forceinline__ void store8(float* p, bool vec, const float (&x)[8]) {
    if (vec) {
      reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = x[j];
    }
  }
};

// Eight consecutive elements as stored; `vec`: the address is aligned to 16 bytes.
template <typename Tag>
__device__ __forceinline__ void fetch8(const typename Tag::elem* p, bool vec, uint4 (&raw)[Row<Tag>::kRaw]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < Row<Tag>::kRaw; ++i) raw[i] = ld_stream(p + i * Tag::kVec);
  } else {
    constexpr int E = Tag::kVec / 4;                  // elements of a word
#pragma unroll
    for (int i = 0; i < Row<Tag>::kRaw; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = i * Tag::kVec + j * E;
        w[j] = Row<Tag>::pack(load_scalar(p, at), E == 2 ? load_scalar(p, at + 1) : 0.f);
      }
      raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}
template <typename Tag>
__device__ __forceinline__ void values8(const uint4 (&raw)[Row<Tag>::kRaw], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < Row<Tag>::kRaw; ++i) {
    float y[Tag::kVec];
    unpack(raw[i], y, Tag{});
#pragma unroll
    for (int j = 0; j < Tag::kVec; ++j) x[i * Tag::kVec + j] = y[j];
  }
}

// Sine and cosine of the fp64 angle a, |a| < 2^45: reduced to |r| <= pi/4 (and 2^-8) by multiples of
// pi/2, whose two terms leave 2^44 * 1.5e-33 away, then the Taylor polynomials (remainders below 5e-17).
__device__ __forceinline__ void turn_of(double a, double& sine, double& cosine) {
  const double n = rint(a * 0.63661977236758134308);
  double r = fma(-n, 1.57079632679489661923, a);
  r = fma(-n, 6.12323399573676603587e-17, r);
  const double q = r * r;
  double s = fma(q, -1.0 / 1307674368000.0, 1.0 / 6227020800.0);
  s = fma(q, s, -1.0 / 39916800.0);
  s = fma(q, s, 1.0 / 362880.0);
  s = fma(q, s, -1.0 / 5040.0);
  s = fma(q, s, 1.0 / 120.0);
  s = fma(q, s, -1.0 / 6.0);
  s = fma(q * r, s, r);
  double c = fma(q, 1.0 / 20922789888000.0, -1.0 / 87178291200.0);
  c = fma(q, c, 1.0 / 479001600.0);
  c = fma(q, c, -1.0 / 3628800.0);
  c = fma(q, c, 1.0 / 40320.0);
  c = fma(q, c, -1.0 / 720.0);
  c = fma(q, c, 1.0 / 24.0);
  c = fma(q, c, -0.5);
  c = fma(q, c, 1.0);
  const int k = (int)((long long)n & 3);
  sine = k & 1 ? c : s;
  cosine = k & 1 ? s : c;
  if (k & 2) sine = -sine;
  if ((k + 1) & 2) cosine = -cosine;
}

// A block scale: the e4m3 value nearest to a >= 0 (ties to even, at most 448) and its code.
__device__ __forceinline__ double e4m3_round(double a, unsigned& code) {
  if (!(a < 448.0)) {
    code = 0x7e;
    return 448.0;
  }
  int e = ((__double2hiint(a) >> 20) & 0x7ff) - 1023;
  e = max(e, -6);
  int q = __double2int_rn(a * __hiloint2double((1023 + 3 - e) << 20, 0));
  if (q == 16) {
    q = 8;
    ++e;
  }
  code = q < 8 ? q : ((e + 7) << 3) | (q - 8);
  return (double)q * __hiloint2double((1023 + e - 3) << 20, 0);
}

// The e2m1 code of magnitude x >= 0 in units of u = s * g: the borders between neighbours are
// 0.25, 0.75, 1.25, 1.75, 2.5, 3.5 and 5 units, a tie going to the even code.
__device__ __forceinline__ unsigned e2m1_code(double x, double u) {
  unsigned c = x > 0.25 * u;
  c += x >= 0.75 * u;
  c += x > 1.25 * u;
  c += x >= 1.75 * u;
  c += x > 2.5 * u;
  c += x >= 3.5 * u;
  c += x > 5.0 * u;
  return c;
}

__device__ __forceinline__ float e2m1_value(unsigned code) {
  const unsigned m = code & 7u;                       // two exponent bits, one mantissa bit
  const float v = m < 2 ? 0.5f * m : __uint_as_float(((m >> 1) + 126u) << 23) * ((m & 1) ? 1.5f : 1.f);
  return code & 8u ? -v : v;
}

// Two values to a byte of codes (lo in the low nibble), two to e4m3 bytes; rounded to nearest
// even, at most the largest.
__device__ __forceinline__ uint32_t codes_of(float lo, float hi) {
  uint32_t d;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ uint32_t scales_of(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float e4m3_value(unsigned code) {  // finite, not negative
  const unsigned e = code >> 3, m = code & 7u;
  return e ? __uint_as_float((e + 120u) << 23 | m << 20) : (float)m * 0.001953125f;
}

// A block's half (elements j0 .. j0+7 of `head`) in fp64, both lanes of the block: eight codes,
// the scale's code in `sc`.  pos < 0 and j < rot together: no rotation.
template <typename Tag>
__device__ __noinline__ uint32_t exact_codes(const typename Tag::elem* head, int j0, int rot, bool interleaved,
                                             int pos, const float* inv_freq, float g, unsigned& sc) {
  const int h = rot >> 1;
  double x[8], top = 0.0;
  for (int e = 0; e < 8; ++e) {
    const int j = j0 + e;
    x[e] = (double)load_scalar(head, j);
    if (j < rot) {
      const bool first = interleaved ? !(j & 1) : j < h;
      const double p = (double)load_scalar(head, interleaved ? j ^ 1 : (first ? j + h : j - h));
      double s, c;
      turn_of((double)pos * (double)__ldg(inv_freq + (interleaved ? j >> 1 : (first ? j : j - h))), s, c);
      x[e] = fma(x[e], c, first ? -(p * s) : p * s);
    }
    top = fmax(top, fabs(x[e]));                              // drops NaN
  }
  top = fmax(top, __shfl_xor_sync(3u << (threadIdx.x & 30), top, 1));
  const double s = e4m3_round(top / (double)g / 6.0, sc), u = s * (double)g;
  uint32_t packed = 0;
  for (int e = 0; e < 8; ++e) {
    unsigned code = s > 0.0 ? e2m1_code(fabs(x[e]), u) : 0u;
    code |= x[e] == x[e] && signbit(x[e]) ? 8u : 0u;
    packed |= code << (4 * e);
  }
  return packed;
}

// How partners are found.
enum { kAnyhow, kByLane, kInterleaved };   // the first for any rows; the others for 16-byte aligned

// Threads of a CTA: few rows to one, for a padding row leaves its warp's place empty until all end.
__host__ __device__ constexpr int block_of(int team) { return team == 32 ? 64 : kThreads; }

template <typename Tag, bool kE2M1, int kMode, int kTeam>
__global__ void __launch_bounds__(block_of(kTeam), kTeam == 32 ? (sizeof(typename Tag::elem) == 2 ? 13 : 10) : 3) append_kernel(const AppendLaunch L) {
  using elem = typename Tag::elem;
  constexpr int kRaw = Row<Tag>::kRaw, kAhead = kMode == kAnyhow ? 1 : Row<Tag>::kAhead;
  extern __shared__ __align__(16) float2 s_all[];     // [teams][rot / 2] (cos, sin)
  const pspec_append_args& a = L.a;
  const int tid = threadIdx.x % kTeam, team = threadIdx.x / kTeam;
  const int h = a.rot >> 1;
  const long long t = (long long)blockIdx.x * (block_of(kTeam) / kTeam) + team;
  float2* s_cs = s_all + team * h;
  if (t >= a.T) return;                               // (whole teams leave)

  const long long slot = __ldg(reinterpret_cast<const long long*>(a.slot_mapping) + t);
  if (slot < 0 || slot >= L.slots) {
    if (tid == 0 && slot != PSPEC_PADDING_SLOT_ID) set_err(a.err, PSPEC_DEVERR_BLOCK_RANGE);
    return;
  }
  const long long block = L.slots <= 0x7fffffff ? (unsigned)slot / (unsigned)a.block_size : slot / a.block_size;
  const long long under = block * a.Hkv * a.block_size + (slot - block * a.block_size);   // of head 0

  const int nl = a.D >> 3;                            // threads per head, eight elements each
  const int groups = kTeam / nl;
  const int hg = tid / nl, j0 = (tid - hg * nl) * 8;
  const bool turns = j0 < a.rot;
  const bool low = j0 < h;                            // (half split) partners lie above
  const int from = (low ? tid + (h >> 3) : tid - (h >> 3)) & 31;

  // Query heads; key, then value heads: each thread has every groups-th from its hg-th on.
  const int total_q = a.q ? a.Hq : 0, total_kv = 2 * a.Hkv;
  const bool mine = hg < groups;
  const elem* qs = static_cast<const elem*>(a.q) + t * a.q_stride + j0;
  const elem* ks = static_cast<const elem*>(a.k) + t * a.k_stride + j0;
  const elem* vs = static_cast<const elem*>(a.v) + t * a.v_stride + j0;
  auto fetch_q = [&](int i0, uint4 (&raw)[kAhead][kRaw]) {
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      const int hd = i0 + hg + b * groups;
      if (mine && hd < total_q) fetch8<Tag>(qs + hd * a.D, kMode != kAnyhow || L.vec_q, raw[b]);
    }
  };
  auto fetch_kv = [&](int i0, uint4 (&raw)[kRaw]) {
    const int hd = i0 + hg;
    if (mine && hd < total_kv)
      fetch8<Tag>(hd < a.Hkv ? ks + hd * a.D : vs + (hd - a.Hkv) * a.D,
                  kMode != kAnyhow || (hd < a.Hkv ? L.vec_k : L.vec_v), raw);
  };
  float4 held[4];            // (kByLane) the coefficients of the thread's elements, for all heads
  // x turned, of the head whose part at j0 is src; the largest magnitudes that entered, added.  Every lane
  // of the warp comes here.
  auto turn = [&](const elem* src, bool wanted, const uint4 (&raw)[kRaw], float (&x)[8]) {
    float p[8], reach = 0.f, most = 0.f;
    if constexpr (kMode == kByLane) {
      // (the sign of the sine with the partners')
      const uint32_t flip = !low ? 0u : (sizeof(elem) == 2 ? 0x80008000u : 0x80000000u);
      uint4 o[kRaw];
#pragma unroll
      for (int i = 0; i < kRaw; ++i)
        o[i] = make_uint4(__shfl_sync(0xffffffffu, raw[i].x, from) ^ flip, __shfl_sync(0xffffffffu, raw[i].y, from) ^ flip,
                          __shfl_sync(0xffffffffu, raw[i].z, from) ^ flip, __shfl_sync(0xffffffffu, raw[i].w, from) ^ flip);
      values8<Tag>(o, p);
    }
    if (!turns || !wanted) return 0.f;
    if constexpr (kMode == kByLane) {                 // whole threads turn
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float4 v = held[e >> 1];
        reach = fmaxf(reach, fmaxf(fabsf(x[e]), fabsf(x[e + 1])));
        most = fmaxf(most, fmaxf(fabsf(p[e]), fabsf(p[e + 1])));
        x[e] = fmaf(x[e], v.x, p[e] * v.y);
        x[e + 1] = fmaf(x[e + 1], v.z, p[e + 1] * v.w);
      }
    } else if (kMode == kInterleaved || a.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        if (j0 + e < a.rot) {
          const float2 v = s_cs[((j0 + e) >> 1)];
          const float u = x[e], w = x[e + 1];
          reach = fmaxf(reach, fmaxf(fabsf(u), fabsf(w)));
          x[e] = fmaf(u, v.x, -(w * v.y));
          x[e + 1] = fmaf(w, v.x, u * v.y);
        }
      }
      most = reach;
    } else {
#pragma unroll 1
      for (int j = j0; j < min(j0 + 8, a.rot); ++j) {
        const bool under = j < h;
        const float2 v = s_cs[(under ? j : j - h)];
        const float u = load_scalar(src, j - j0), w = load_scalar(src, (under ? j + h : j - h) - j0);
        reach = fmaxf(reach, fabsf(u));
        most = fmaxf(most, fabsf(w));
        const float y = fmaf(u, v.x, w * (under ? -v.y : v.y));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = j0 + e == j ? y : x[e];
      }
    }
    return reach + most;
  };

  uint4 raw[kAhead][kRaw] = {}, next[2][kRaw] = {};   // key and value heads two ahead
  fetch_kv(0, next[0]);
  fetch_kv(groups, next[1]);
  fetch_q(0, raw);

  const double pos = (double)__ldg(a.positions + t);
  for (int j = tid; j < h; j += kTeam) {
    double s, c;
    turn_of(pos * (double)__ldg(a.inv_freq + j), s, c);
    s_cs[j] = make_float2((float)c, (float)s);
  }
  if constexpr (kTeam == 32) __syncwarp();
  else __syncthreads();

  if constexpr (kMode == kByLane) {
    const float4* cs = reinterpret_cast<const float4*>(s_cs + (low ? j0 : j0 - h));
#pragma unroll
    for (int i = 0; i < 4; ++i) held[i] = turns ? cs[i] : make_float4(1.f, 0.f, 1.f, 0.f);
  }
  elem* qo = static_cast<elem*>(a.q_out) + t * a.Hq * a.D + j0;
  for (int i0 = 0; i0 < total_q; i0 += kAhead * groups) {     // the same for every thread
    if (i0 > 0) fetch_q(i0, raw);
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      const int hd = i0 + hg + b * groups;
      const bool ok = mine && hd < total_q;
      float x[8];
      values8<Tag>(raw[b], x);
      turn(qs + hd * a.D, ok, raw[b], x);
      if (ok) Row<Tag>::store8(qo + hd * a.D, kMode != kAnyhow || L.vec_qo, x);
    }
  }

#pragma unroll 1
  for (int i0 = 0; i0 < total_kv; i0 += groups) {
    const bool ok = mine && i0 + hg < total_kv, is_k = i0 + hg < a.Hkv;
    const int hd = is_k ? i0 + hg : i0 + hg - a.Hkv;
    const elem* src = (is_k ? ks : vs) + hd * a.D;
    float x[8];
    values8<Tag>(next[0], x);
    const float reach = turn(src, ok && is_k, next[0], x);
#pragma unroll
    for (int i = 0; i < kRaw; ++i) next[0][i] = next[1][i];
    fetch_kv(i0 + 2 * groups, next[1]);
    if (!ok) continue;
    elem* echo_all = static_cast<elem*>(is_k ? a.k_out : a.v_out);
    const bool vec_e = kMode != kAnyhow || (is_k ? L.vec_ko : L.vec_vo);
    const long long row = under + (long long)hd * a.block_size;      // row of the cache
    elem* echo = echo_all ? echo_all + (t * a.Hkv + hd) * a.D + j0 : nullptr;
    if constexpr (!kE2M1) {
      Row<Tag>::store8(static_cast<elem*>(is_k ? a.k_pages : a.v_pages) + row * a.D + j0, true, x);
      if (echo) Row<Tag>::store8(echo, vec_e, x);
    } else {
      const unsigned pair = 3u << (threadIdx.x & 30);
      // |fp32 value - exact value| <= err: the coefficients are off by 2^-24, products and sum
      // rounded, 2.5 * 2^-24 of the two magnitudes; 2^-20 leaves room
      float err = reach * 9.5367432e-7f, top = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));   // drops NaN
      top = fmaxf(top, __shfl_xor_sync(pair, top, 1));
      const float err2 = fmaxf(err, __shfl_xor_sync(pair, err, 1));
      const float* scales = is_k ? a.k_scale : a.v_scale;
      const float g = scales ? __ldg(scales + hd) : 1.f;
      // the scale from both ends of its interval (the quotients are off by 2^-21 at most)
      const float per6 = 1.f / (6.f * g), mid = top * per6;
      const float wide = fmaf(mid, 1e-6f, err2 * per6);
      const unsigned ends = scales_of(fmaxf(mid - wide, 0.f), mid + wide);
      unsigned sc = ends & 0xffu;
      const float s = e4m3_value(sc), per = s > 0.f ? 1.f / (s * g) : 0.f;
      uint32_t packed = 0;
      // (far from 1 a head scale takes the quotients, and a small rotated value its error, out of fp32's
      // normal range, where the interval no longer holds the exact value)
      bool sure = ends == sc * 0x101u && wide <= 1e30f && g > 1e-20f && g < 1e20f && (reach == 0.f || reach > 1e-30f);
      const float room = err * per;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float z0 = x[2 * c] * per, z1 = x[2 * c + 1] * per;
        const float w0 = fmaf(fabsf(z0), 1e-6f, room), w1 = fmaf(fabsf(z1), 1e-6f, room);
        const uint32_t lo = codes_of(z0 - w0, z1 - w1), hi = codes_of(z0 + w0, z1 + w1);
        // (NaN, and the sign of a zero that may be either side: not sure)
        sure = sure && lo == hi && z0 == z0 && z1 == z1;
        packed |= lo << (8 * c);
      }
      sure = __shfl_xor_sync(pair, sure, 1) && sure;
      if (!sure)
        packed = exact_codes<Tag>(src - j0, j0, is_k ? a.rot : 0, a.interleaved != 0, __ldg(a.positions + t), a.inv_freq, g, sc);
      uint8_t* pages = static_cast<uint8_t*>(is_k ? a.k_pages : a.v_pages);
      *reinterpret_cast<uint32_t*>(pages + row * (a.D >> 1) + (j0 >> 1)) = packed;
      if ((j0 & 15) == 0) {
        uint8_t* bs = static_cast<uint8_t*>(is_k ? a.k_block_scales : a.v_block_scales);
        bs[row * (a.D >> 4) + (j0 >> 4)] = (uint8_t)sc;
      }
      if (echo) {                                 // level * s is exact, one rounding with g
        const float sv = e4m3_value(sc);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e2m1_value(packed >> (4 * e)) * sv * g;
        Row<Tag>::store8(echo, vec_e, v);
      }
    }
  }
}

template <typename Tag>
void launch_rows(const AppendLaunch& L, cudaStream_t stream) {
  const pspec_append_args& a = L.a;
  // A CTA to a row while there are few, else a warp: rows then wait for nothing but their own
  // loads (15360 rows, both as first built: 83 us, by CTAs of four rows 101).
  const bool warps = a.T > 8 * kNumSMs && a.D <= 256;
  const int teams = warps ? block_of(32) / 32 : 1;
  const unsigned grid = (unsigned)(((long long)a.T + teams - 1) / teams);
  const size_t smem = (size_t)teams * (a.rot / 2) * sizeof(float2);
  const bool aligned = (!a.q || (L.vec_q && L.vec_qo)) && L.vec_k && L.vec_v && L.vec_ko && L.vec_vo;
  // partners in another lane: a head's lanes lie in one warp, whole threads on each side
  const int nl = a.D / 8;
  int mode = kAnyhow;
  if (aligned && a.rot == 0) mode = kInterleaved;
  else if (aligned && a.interleaved) mode = kInterleaved;
  else if (aligned && (nl & (nl - 1)) == 0 && nl <= 32 && a.rot % 16 == 0) mode = kByLane;
  auto go = [&](auto* one, auto* many) {
    if (warps) many<<<grid, block_of(32), smem, stream>>>(L);
    else one<<<grid, kThreads, smem, stream>>>(L);
  };
  auto pick = [&](auto e2m1) {
    constexpr bool kE2M1 = decltype(e2m1)::value;
    if (mode == kByLane) go(append_kernel<Tag, kE2M1, kByLane, kThreads>, append_kernel<Tag, kE2M1, kByLane, 32>);
    else if (mode == kInterleaved) go(append_kernel<Tag, kE2M1, kInterleaved, kThreads>, append_kernel<Tag, kE2M1, kInterleaved, 32>);
    else go(append_kernel<Tag, kE2M1, kAnyhow, kThreads>, append_kernel<Tag, kE2M1, kAnyhow, 32>);
  };
  if (a.cache == PSPEC_CACHE_E2M1) pick(std::true_type{});
  else pick(std::false_type{});
}

}  // namespace

cudaError_t launch_append(const AppendLaunch& L, cudaStream_t stream) {
  if (L.a.dtype == PSPEC_BF16) launch_rows<BF16Tag>(L, stream);
  else launch_rows<F32Tag>(L, stream);
  return cudaGetLastError();
}

}  // namespace pspec
