// attend_common.cuh -- what the kernels of attention over the 4-bit cache share: the list of work,
// rows and keys made safe, conversions, and the last step of an output row.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "plan.h"

namespace pspec {

namespace attention {

constexpr int kUnit = 64;                       // keys of one unit of work
// Probabilities are formed as 2^(x - m + kShift) and the maximum m follows only when a row
// passes it by more than kSlack: both leave them below 2^15 (fp16 holds 65504) and far above
// fp16's subnormals, and the outputs are rescaled rarely.
constexpr float kShift = 7.f, kSlack = 8.f;
// An exponent x - m + kShift is one fused operation on the score, which does not round the product x;
// the maximum m is a product rounded.  From 2^24 on the two differ by whole octaves (from 2^27: by
// more than fp16 holds), so where a row has come so far both are rounded, in a second go over the unit.
constexpr float kCoarse = 16777216.f;

// Four bytes of two e2m1 codes each, as four fp16 pairs (low nibble first).
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t scales_to_half(uint32_t two) {   // two e4m3 bytes
  uint32_t h;
  // the maximum with zero: a NaN scale (a key that no row may see can hold anything) or a
  // negative one counts as 0, so that a probability of zero times the value is zero
  asm("{\n\t.reg .b16 s;\n\t.reg .b32 v;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 v, s;\n\t"
      "max.f16x2 %0, v, %2;\n\t}" : "=r"(h) : "r"(two), "r"(0u));
  return h;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float half_lo(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h));
  return f;
}
__device__ __forceinline__ float half_hi(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, u;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

// The rows and keys of sequence i, made safe: a malformed offset pair has no rows, lengths
// stay inside the block table.
struct Seq {
  int row0, rows, len, tiles;
  long long units;     // of one tile
  int err;
};

template <int kTileRows>
__device__ __forceinline__ Seq seq_of(const pspec_attend_args& a, int i, int group) {
  Seq s;
  s.err = 0;
  const int lo = __ldg(a.qsl + i), hi = __ldg(a.qsl + i + 1);
  s.row0 = lo;
  s.rows = hi - lo;
  if (lo < 0 || hi < lo || hi > a.T) {
    s.err |= PSPEC_DEVERR_LAYOUT;
    s.row0 = s.rows = 0;
  }
  const long long room = (long long)a.max_blocks * a.block_size;
  s.len = __ldg(a.seq_lens + i);
  if (s.len < 0 || s.len > room) {
    s.err |= PSPEC_DEVERR_BLOCK_RANGE;
    s.len = s.len < 0 ? 0 : (int)room;
  }
  const long long n = (long long)s.rows * group;
  s.tiles = (int)((n + kTileRows - 1) / kTileRows);
  s.units = s.len == 0 ? 1 : ((long long)s.len + kUnit - 1) / kUnit;   // an empty tile is a unit too
  return s;
}

// Row r of a tile's sequence: its token, query head and the number of keys it may see (-1: the
// row is not computed).
struct RowRef {
  long long at;        // token * Hq + head
  int limit;
};

__device__ __forceinline__ RowRef row_of(const pspec_attend_args& a, const Seq& s, int group, int h,
                                         long long r) {
  RowRef x{0, -1};
  if (r >= (long long)s.rows * group) return x;
  const int j = (int)(r / group);
  const int t = s.row0 + j;
  if (a.row_kind && __ldg(a.row_kind + t) >= PSPEC_ROW_REJ) return x;
  x.at = (long long)t * a.Hq + h * group + (int)(r - (long long)j * group);
  const int pos = __ldg(a.positions + t);
  x.limit = pos < 0 ? 0 : min(s.len, pos == 0x7fffffff ? pos : pos + 1);
  return x;
}

// The factor of a row's scores in base 2, its queries having been multiplied by 2^up.  The head scale
// meets that power first: each may lie where its product with another factor would leave fp32.
__device__ __forceinline__ float score_factor(float scale, float kscale, int up) {
  return scale * kLog2e * (kscale * __uint_as_float((unsigned)(127 - up) << 23));
}

__device__ __forceinline__ void load_q2(const uint16_t* p, float& x, float& y) {
  x = __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
  y = __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + 1) << 16);
}
__device__ __forceinline__ void load_q2(const float* p, float& x, float& y) {
  x = __ldg(p);
  y = __ldg(p + 1);
}

__device__ __forceinline__ void store_out(uint16_t* p, float4 v) {
  uint32_t lo, hi;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(v.y), "f"(v.x));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(v.w), "f"(v.z));
  *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
}
__device__ __forceinline__ void store_out(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

// Where a key lies: its page's column of the block table and its place in the page.
struct Walk {
  int col, off;
  __device__ __forceinline__ void set(long long key, int block_size) {
    col = (int)((unsigned)key / (unsigned)block_size);
    off = (int)((unsigned)key - (unsigned)col * (unsigned)block_size);
  }
  __device__ __forceinline__ void advance(int cols, int rest, int block_size) {   // by a unit
    col += cols;
    off += rest;
    if (off >= block_size) {
      off -= block_size;
      ++col;
    }
  }
};

// A CTA's share [w0, w1) of the list of units -- all units of all tiles of all kv heads of all
// sequences in this order -- and the sequence where it begins, whose first unit is `prefix`.
struct Share {
  long long U, E;      // units of all, CTAs with a share
  long long w0, w1, prefix;
  int seq;
};
struct ShareSmem {
  long long scan[32];
  int seq;
  long long prefix;
};

// Every thread of the CTA; false when there is none for it.  CTA 0 reports the sequences' errors.
template <int kTileRows, int kThreadsN>
__device__ __forceinline__ bool share_of(const pspec_attend_args& a, int group, int ctas, ShareSmem& sm, Share& x) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  const int per = (a.B + kThreadsN - 1) / kThreadsN;
  const int i_lo = min(a.B, tid * per), i_hi = min(a.B, i_lo + per);
  long long mine = 0;
  int bits = 0;
  for (int i = i_lo; i < i_hi; ++i) {
    const Seq s = seq_of<kTileRows>(a, i, group);
    mine += s.units * s.tiles * a.Hkv;
    bits |= s.err;
  }
  if (cta == 0) set_err(a.err, bits);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) sm.scan[warp] = incl;
  __syncthreads();
  long long base = 0;
  x.U = 0;
  for (int w = 0; w < kThreadsN / 32; ++w) {
    if (w < warp) base += sm.scan[w];
    x.U += sm.scan[w];
  }
  x.E = min((long long)ctas, x.U);
  if (cta >= x.E) return false;
  x.w0 = cta * x.U / x.E;
  x.w1 = (cta + 1) * x.U / x.E;
  long long at = base + incl - mine;
  if (x.w0 >= at && x.w0 < at + mine) {
    for (int i = i_lo; i < i_hi; ++i) {
      const Seq s = seq_of<kTileRows>(a, i, group);
      const long long n = s.units * s.tiles * a.Hkv;
      if (x.w0 < at + n) {
        sm.seq = i;
        sm.prefix = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  x.seq = sm.seq;
  x.prefix = sm.prefix;
  return true;
}

// Four columns of an output row from its sum of values v, sum of probabilities and maximum.
template <int D, typename elem>
__device__ __forceinline__ void finish_row(const pspec_attend_args& a, const RowRef& rr, int d, float M, float sum,
                                           float vscale, float4 v) {
  if (rr.limit < 0) return;
  float f = sum > 0.f ? vscale / sum : (sum == 0.f ? 0.f : sum), g = 1.f;
  if (f < 1e-37f && sum > 0.f) {                  // a quotient below fp32's normal range: in two factors
    f = 1.f / sum;
    g = vscale;
  }
  store_out(static_cast<elem*>(a.out) + rr.at * D + d, make_float4(v.x * f * g, v.y * f * g, v.z * f * g, v.w * f * g));
  if (a.lse && d == 0)
    a.lse[rr.at] = sum == 0.f ? -INFINITY : (M - kShift + log2f(sum)) * 0.69314718055994530942f;
}

}  // namespace attention
}  // namespace pspec
