// attend.cu -- attention of a ragged batch over the 4-bit paged cache (one launch).
//
// Work: a tile is up to 16 query rows (token x head of the group) of one sequence and kv head;
// its keys are cut into units of 64.  All units of all tiles form one list, dealt out evenly
// to persistent CTAs, so ragged lengths cost no balance and neither grid nor workspace depends
// on them.  A CTA's share covers at most two tiles partly (its first and its last); those go to
// the workspace as (max, sum, unnormalised output), and the CTA that arrives last joins them
// in key order.
//
// Per unit each of the four warps takes 16 keys and keeps its own running maximum and sum, so
// the loop has no barrier.  The cache's bytes come by asynchronous copies into a ring of the
// warp's own.  A dot product may run over the head dimension in any order, and a sum over keys
// in any order of keys, so the fragments of the fp16 tensor-core products are laid to the
// cache's bytes instead of the other way round: a lane's 16 (or 8) bytes of one key ARE its
// fragments of 8 (or 4) products, and two keys' nibbles interleaved are the pairs that the
// product with the values wants.  Dequantised values are exact in fp16: 2 significant bits of
// the code times 4 of the scale, between 2^-10 and 2688.
#include "common.cuh"
#include "kernels.h"
#include "plan.h"

namespace pspec {

namespace {

constexpr int kAttWarps = 4;
constexpr int kAttThreads = 32 * kAttWarps;
constexpr int kStep = 16;                       // keys of one warp step
constexpr int kUnit = kStep * kAttWarps;        // keys of one unit
constexpr int kTileRows = 16;
constexpr int kStages = 4;
constexpr int kAttendMaxCtas = kNumSMs * 4;
// Probabilities are formed as 2^(x - m + kShift) and the maximum m follows only when a row
// passes it by more than kSlack: both leave them below 2^15 (fp16 holds 65504) and far above
// fp16's subnormals, and the outputs are rescaled rarely.
constexpr float kShift = 7.f, kSlack = 8.f;

template <int D>
struct Shape {
  static constexpr int kLane = D / 4;           // values of a key that a lane holds
  static constexpr int kWords = D / 32;         // their 32-bit words
  static constexpr int kK = D / 16;             // products over the head dimension
  static constexpr int kCols = D / 8;           // output columns per column group
  static constexpr int kRow = D / 2;            // bytes of a key
  static constexpr int kScaleRow = D / 16;
  static constexpr int kStage = 2 * kStep * (kRow + kScaleRow);
  static constexpr int kRing = kStages * kStage;
  static constexpr long long kPart = kTileRows * (D + 2);   // floats of a partial tile
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0));
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(live ? N : 0));
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

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

template <int D, typename Tag>
struct AttendSmem {
  union {
    alignas(128) uint8_t ring[kAttWarps][Shape<D>::kRing];
    float out[kAttWarps][kTileRows][D + 4];
  };
  float m[kAttWarps][kTileRows];
  float l[kAttWarps][kTileRows];
  unsigned live[kAttWarps][kStages];          // which of the stage's keys exist
  long long scan[kAttWarps];
  int start_seq;
  long long start_prefix;
  int last;
};

template <int D, typename Tag, bool kWholePages>
__global__ void __launch_bounds__(kAttThreads, sizeof(typename Tag::elem) == 2 ? 3 : 2)
attend_kernel(const AttendLaunch L) {
  using elem = typename Tag::elem;
  using S = Shape<D>;
  constexpr bool kF32 = sizeof(elem) == 4;     // two fp16 terms for queries and probabilities
  extern __shared__ __align__(128) uint8_t s_raw[];
  auto& sm = *reinterpret_cast<AttendSmem<D, Tag>*>(s_raw);
  const pspec_attend_args& a = L.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int group = a.Hq / a.Hkv;
  const int cta = blockIdx.x;

  // ---- the list of units: its length, and the sequence where this CTA's share begins
  const int per = (a.B + kAttThreads - 1) / kAttThreads;
  const int i_lo = min(a.B, tid * per), i_hi = min(a.B, i_lo + per);
  long long mine = 0;
  int bits = 0;
  for (int i = i_lo; i < i_hi; ++i) {
    const Seq s = seq_of(a, i, group);
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
  long long base = 0, U = 0;
  for (int w = 0; w < kAttWarps; ++w) {
    if (w < warp) base += sm.scan[w];
    U += sm.scan[w];
  }
  const long long E = min((long long)L.ctas, U);            // CTAs with a share
  if (cta >= E) return;
  const long long w0 = cta * U / E, w1 = (cta + 1) * U / E;
  {
    long long at = base + incl - mine;
    if (w0 >= at && w0 < at + mine) {
      for (int i = i_lo; i < i_hi; ++i) {
        const Seq s = seq_of(a, i, group);
        const long long n = s.units * s.tiles * a.Hkv;
        if (w0 < at + n) {
          sm.start_seq = i;
          sm.start_prefix = at;
          break;
        }
        at += n;
      }
    }
  }
  __syncthreads();
  int seq = sm.start_seq;
  long long prefix = sm.start_prefix;

  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm.ring[warp]);
  const uint8_t* ring_p = sm.ring[warp];
  // shared-memory offsets of the lane's bytes: key tau of tile j is 8 j + (g even ? g/2 :
  // 7 - g/2), so that the keys of a lane's value pairs are t, 7-t, 8+t and 15-t; 16-byte
  // chunks of odd key pairs are swapped by two (D = 128) to keep the reads free of conflicts
  const int tau = (g & 1) ? 7 - (g >> 1) : g >> 1;

  long long w = w0;
  bool first = true;
  Seq s = seq_of(a, seq, group);
  while (w < w1) {
    while (w >= prefix + s.units * s.tiles * a.Hkv) {
      prefix += s.units * s.tiles * a.Hkv;
      s = seq_of(a, ++seq, group);
    }
    const long long item = (w - prefix) / s.units;
    const long long item0 = prefix + item * s.units;          // the tile's first unit
    const int h = (int)(item / s.tiles);
    const long long r0 = (item - (long long)h * s.tiles) * kTileRows;
    const long long u0 = w - item0;
    const long long u1 = min(s.units, w1 - item0);
    w = item0 + u1;

    const RowRef ra = row_of(a, s, group, h, r0 + g), rb = row_of(a, s, group, h, r0 + g + 8);
    int lim_hi = max(ra.limit, rb.limit);
    int lim_lo = min(ra.limit < 0 ? 0x7fffffff : ra.limit, rb.limit < 0 ? 0x7fffffff : rb.limit);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      lim_hi = max(lim_hi, __shfl_xor_sync(0xffffffffu, lim_hi, o));
      lim_lo = min(lim_lo, __shfl_xor_sync(0xffffffffu, lim_lo, o));
    }
    const int* table = a.block_table + (long long)seq * a.max_blocks;
    const int steps = (int)(min(u1, ((long long)max(lim_hi, 0) + kUnit - 1) / kUnit) - u0);

    // ---- one step's copies; `blk` is the page of a step inside one page
    auto block_of = [&](long long key) -> int {
      return key < s.len ? __ldg(table + (unsigned)key / (unsigned)a.block_size) : -1;
    };
    auto issue = [&](int step, int blk) {
      const long long k0 = (u0 + step) * kUnit + warp * kStep;
      const uint32_t dst = ring + (step % kStages) * S::kStage;
      auto row_at = [&](int key, bool& live) -> long long {     // row of the cache
        const long long k = k0 + key;
        int b = blk;
        if constexpr (!kWholePages) b = block_of(k);
        live = k < s.len && b >= 0 && b < a.num_blocks;
        if (!live) return 0;
        return ((long long)b * a.Hkv + h) * a.block_size + (int)((unsigned)k % (unsigned)a.block_size);
      };
      bool live;
      if constexpr (D == 128) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int key = (lane >> 2) + 8 * half, c = lane & 3;
          const long long row = row_at(key, live) * S::kRow + c * 16;
          const uint32_t to = dst + key * S::kRow + ((c ^ ((key >> 1 & 1) << 1)) << 4);
          cp_async16(to, static_cast<const uint8_t*>(a.k_pages) + row, live);
          cp_async16(to + kStep * S::kRow, static_cast<const uint8_t*>(a.v_pages) + row, live);
        }
      } else {
        const int key = lane >> 1, c = lane & 1;
        const long long row = row_at(key, live) * S::kRow + c * 16;
        const uint32_t to = dst + key * S::kRow + (c << 4);
        cp_async16(to, static_cast<const uint8_t*>(a.k_pages) + row, live);
        cp_async16(to + kStep * S::kRow, static_cast<const uint8_t*>(a.v_pages) + row, live);
      }
      const int key = lane & 15;
      const long long row = row_at(key, live) * S::kScaleRow;
      const void* src = static_cast<const uint8_t*>(lane < 16 ? a.k_block_scales : a.v_block_scales) + row;
      cp_async_small<S::kScaleRow>(dst + 2 * kStep * S::kRow + lane * S::kScaleRow, src, live);
      const unsigned alive = __ballot_sync(0xffffffffu, live) & 0xffffu;
      if (lane == 0) {
        sm.live[warp][step % kStages] = alive;
        // a key that exists but whose page does not is hidden
        const int there = (int)max(0LL, min((long long)kStep, s.len - k0));
        if (alive != (1u << there) - 1u) set_err(a.err, PSPEC_DEVERR_BLOCK_RANGE);
      }
    };
    int next_blk = -1;
    if (kWholePages) next_blk = block_of(u0 * kUnit + warp * kStep);
    auto issue_next = [&](int step) {
      if (step < steps) {
        const int blk = next_blk;
        if (kWholePages) next_blk = block_of((u0 + step + 1) * kUnit + warp * kStep);
        issue(step, blk);
      }
      asm volatile("cp.async.commit_group;");
    };
    for (int st = 0; st < kStages - 1; ++st) issue_next(st);

    // ---- the query rows as fragments: power-of-two scaled into fp16's range
    uint32_t qa[S::kK][4], ql[kF32 ? S::kK : 1][4];
    float mult[2];
    {
      const float ks = a.k_scale ? __ldg(a.k_scale + h) : 1.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const RowRef& rr = half ? rb : ra;
        float x[S::kLane];
        float top = 0.f;
        const long long tok = rr.at / a.Hq;
        const elem* p = static_cast<const elem*>(a.q) + tok * a.q_stride + (rr.at - tok * a.Hq) * D + t * S::kLane;
#pragma unroll
        for (int j = 0; j < S::kLane; j += 2) {
          x[j] = x[j + 1] = 0.f;
          if (rr.limit > 0) load_q2(p + j, x[j], x[j + 1]);
          top = fmaxf(top, fmaxf(fabsf(x[j]), fabsf(x[j + 1])));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^(14 - exponent of the row's largest element), kept within fp32's normal range
        const int ex = (int)(__float_as_uint(top) >> 23) - 127;
        const int up = top == 0.f || ex == 128 ? 0 : min(100, 14 - ex);
        const float f = __uint_as_float((unsigned)(127 + up) << 23);
        mult[half] = a.scale * kLog2e * ks * __uint_as_float((unsigned)(127 - up) << 23);
#pragma unroll
        for (int k = 0; k < S::kK; ++k)
#pragma unroll
          for (int pair = 0; pair < 2; ++pair) {
            const float u = x[4 * k + 2 * pair] * f, v = x[4 * k + 2 * pair + 1] * f;
            const uint32_t hi = pack_half(u, v);
            qa[k][2 * pair + half] = hi;
            if constexpr (kF32) ql[k][2 * pair + half] = pack_half(u - half_lo(hi), v - half_hi(hi));
          }
      }
    }

    float o[S::kCols][4];
#pragma unroll
    for (int j = 0; j < S::kCols; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[j][c] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int step = 0; step < steps; ++step) {
      issue_next(step + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1));
      __syncwarp();
      const uint8_t* buf = ring_p + (step % kStages) * S::kStage;
      const long long k0 = (u0 + step) * kUnit + warp * kStep;
      const unsigned alive = sm.live[warp][step % kStages];

      // ---- scores: 16 rows x 16 keys
      float sc[2][4] = {};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int key = 8 * j + tau;
        uint32_t wd[S::kWords];
        if constexpr (D == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(buf + key * S::kRow + ((t ^ ((key >> 1 & 1) << 1)) << 4));
          wd[0] = v.x; wd[1] = v.y; wd[2] = v.z; wd[3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(buf + key * S::kRow + t * 8);
          wd[0] = v.x; wd[1] = v.y;
        }
        const uint8_t* sp = buf + 2 * kStep * S::kRow + key * S::kScaleRow;
        uint32_t s_lo, s_hi;
        if constexpr (D == 128) {
          const uint32_t two = scales_to_half(*reinterpret_cast<const uint16_t*>(sp + 2 * t));
          s_lo = __byte_perm(two, 0, 0x1010);
          s_hi = __byte_perm(two, 0, 0x3232);
        } else {
          const uint32_t one = sp[t];
          s_lo = s_hi = scales_to_half(one | one << 8);
        }
#pragma unroll
        for (int k = 0; k < S::kWords; ++k) {
          uint32_t b[4];
          codes_to_half(wd[k], b);
          const uint32_t f = 2 * k < S::kWords ? s_lo : s_hi;
#pragma unroll
          for (int i = 0; i < 4; ++i) b[i] = hmul2(b[i], f);
          mma16816(sc[j], qa[2 * k], b[0], b[1]);
          mma16816(sc[j], qa[2 * k + 1], b[2], b[3]);
          if constexpr (kF32) {
            mma16816(sc[j], ql[2 * k], b[0], b[1]);
            mma16816(sc[j], ql[2 * k + 1], b[2], b[3]);
          }
        }
      }

      // ---- softmax in base 2; a lane's columns of tile j are keys 8j + t and 8j + 7 - t
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[j][c] *= mult[c >> 1];
      if (alive != 0xffffu || k0 + kStep > lim_lo) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = 8 * j + ((c & 1) ? 7 - t : t);
            if (!(alive >> key & 1) || k0 + key >= (c >> 1 ? rb.limit : ra.limit)) sc[j][c] = -INFINITY;
          }
      }
      float top[2];
      bool grow = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        top[r] = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
        grow |= top[r] > m[r] + kSlack;
      }
      if (__any_sync(0xffffffffu, grow)) {
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float n = fmaxf(m[r], top[r]);
          f[r] = n == -INFINITY ? 1.f : ex2(m[r] - n);
          m[r] = n;
          l[r] *= f[r];
        }
#pragma unroll
        for (int j = 0; j < S::kCols; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[j][c] *= f[c >> 1];
      }
      uint32_t pa[4], pl[4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float at = m[r] == -INFINITY ? 0.f : m[r] - kShift;
          const float x = ex2(sc[j][2 * r] - at), y = ex2(sc[j][2 * r + 1] - at);
          l[r] += x + y;
          const uint32_t hi = pack_half(x, y);
          pa[2 * j + r] = hi;
          if constexpr (kF32) pl[2 * j + r] = pack_half(x - half_lo(hi), y - half_hi(hi));
        }

      // ---- outputs: pairs of keys (t, 7 - t) and (8 + t, 15 - t)
      const uint8_t* vb = buf + kStep * S::kRow;
      const uint8_t* vs = buf + 2 * kStep * S::kRow + kStep * S::kScaleRow;
      const int key[4] = {t, 7 - t, 8 + t, 15 - t};
      uint32_t vw[4][D / 64];
      uint32_t f[2];
      {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) {
            const uint2 v = *reinterpret_cast<const uint2*>(
                vb + key[i] * S::kRow + (((g >> 1) ^ ((key[i] >> 1 & 1) << 1)) << 4) + (g & 1) * 8);
            vw[i][0] = v.x;
            vw[i][1] = v.y;
            b[i] = vs[key[i] * S::kScaleRow + g];
          } else {
            vw[i][0] = *reinterpret_cast<const uint32_t*>(vb + key[i] * S::kRow + g * 4);
            b[i] = vs[key[i] * S::kScaleRow + (g >> 1)];
          }
        }
        f[0] = scales_to_half(b[0] | b[1] << 8);
        f[1] = scales_to_half(b[2] | b[3] << 8);
      }
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {                 // even, then odd columns of the word
          uint32_t b0[4], b1[4];
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            const uint32_t x = vw[2 * pr][k], y = vw[2 * pr + 1][k];
            const uint32_t both = odd ? ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u)
                                      : (x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u);
            if (pr == 0) codes_to_half(both, b0);
            else codes_to_half(both, b1);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = hmul2(b0[i], f[0]), y = hmul2(b1[i], f[1]);
            mma16816(o[8 * k + 2 * i + odd], pa, x, y);
            if constexpr (kF32) mma16816(o[8 * k + 2 * i + odd], pl, x, y);
          }
        }
      }
      __syncwarp();                                         // the stage may be refilled
    }
    asm volatile("cp.async.wait_group 0;");
    __syncthreads();                                        // every warp is done with its ring

    // ---- the four warps' results joined
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      const int row = g + 8 * r;
      if (t == 0) {
        sm.m[warp][row] = m[r];
        sm.l[warp][row] = l[r];
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)                           // column group 2t + n
#pragma unroll
        for (int j = 0; j < S::kCols; j += 4)
          *reinterpret_cast<float4*>(&sm.out[warp][row][S::kCols * (2 * t + n) + j]) =
              make_float4(o[j][2 * r + n], o[j + 1][2 * r + n], o[j + 2][2 * r + n], o[j + 3][2 * r + n]);
    }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == s.units;
    float* part = L.parts + (2LL * cta + (first ? 0 : 1)) * S::kPart;
    first = false;
    const float vscale = a.v_scale ? __ldg(a.v_scale + h) : 1.f;
    elem* out = static_cast<elem*>(a.out);

    auto finish = [&](const RowRef& rr, int d, float M, float l_sum, float4 v) {
      if (rr.limit < 0) return;
      const float f = l_sum > 0.f ? vscale / l_sum : (l_sum == 0.f ? 0.f : l_sum);
      store_out(out + rr.at * D + d, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
      if (a.lse && d == 0)
        a.lse[rr.at] = l_sum == 0.f ? -INFINITY : (M - kShift + log2f(l_sum)) * 0.69314718055994530942f;
    };

    for (int i = tid; i < kTileRows * (D / 4); i += kAttThreads) {
      const int row = i / (D / 4), d = (i - row * (D / 4)) * 4;
      float M = sm.m[0][row];
#pragma unroll
      for (int x = 1; x < kAttWarps; ++x) M = fmaxf(M, sm.m[x][row]);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int x = 0; x < kAttWarps; ++x) {
        const float f = sm.m[x][row] == -INFINITY ? 0.f : ex2(sm.m[x][row] - M);
        const float4 p = *reinterpret_cast<const float4*>(&sm.out[x][row][d]);
        sum += f * sm.l[x][row];
        v.x += f * p.x; v.y += f * p.y; v.z += f * p.z; v.w += f * p.w;
      }
      if (whole) {
        finish(row_of(a, s, group, h, r0 + row), d, M, sum, v);
      } else {
        *reinterpret_cast<float4*>(part + row * D + d) = v;
        if (d == 0) {
          part[kTileRows * D + row] = M;
          part[kTileRows * D + kTileRows + row] = sum;
        }
      }
    }
    if (!whole) {
      // the tile's CTAs are the ones whose shares hold its first and last unit and all between
      const long long cta_a = ((item0 + 1) * E - 1) / U;
      const long long cta_b = ((item0 + s.units) * E - 1) / U;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int n = atomicAdd(L.cnt + cta_a, 1) + 1;
        sm.last = n == (int)(cta_b - cta_a + 1);
        if (sm.last) L.cnt[cta_a] = 0;
      }
      __syncthreads();
      if (sm.last) {
        __threadfence();
        // in CTA a the tile is the first of the share only when it begins there
        const long long slot_a = 2 * cta_a + (cta_a * U / E == item0 ? 0 : 1);
        for (int i = tid; i < kTileRows * (D / 4); i += kAttThreads) {
          const int row = i / (D / 4), d = (i - row * (D / 4)) * 4;
          const RowRef rr = row_of(a, s, group, h, r0 + row);
          if (rr.limit < 0) continue;
          float M = -INFINITY;
          for (long long c = cta_a; c <= cta_b; ++c) {
            const float* p = L.parts + (c == cta_a ? slot_a : 2 * c) * S::kPart;
            M = fmaxf(M, ld_cg(p + kTileRows * D + row));
          }
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          float sum = 0.f;
          for (long long c = cta_a; c <= cta_b; ++c) {
            const float* p = L.parts + (c == cta_a ? slot_a : 2 * c) * S::kPart;
            const float mc = ld_cg(p + kTileRows * D + row);
            const float f = mc == -INFINITY ? 0.f : ex2(mc - M);
            const float4 x = ld_cg(reinterpret_cast<const float4*>(p + row * D + d));
            sum += f * ld_cg(p + kTileRows * D + kTileRows + row);
            v.x += f * x.x; v.y += f * x.y; v.z += f * x.z; v.w += f * x.w;
          }
          finish(rr, d, M, sum, v);
        }
      }
    }
    __syncthreads();                                        // shared memory is the ring's again
  }
}

template <int D, typename Tag>
cudaError_t launch_d(const AttendLaunch& L, cudaStream_t stream) {
  constexpr int smem = sizeof(AttendSmem<D, Tag>);
  const bool whole = L.a.block_size % kStep == 0;
  auto* fn = whole ? attend_kernel<D, Tag, true> : attend_kernel<D, Tag, false>;
  static_assert(smem <= 48 * 1024, "within the default limit");
  fn<<<L.ctas, kAttThreads, smem, stream>>>(L);
  return cudaGetLastError();
}

}  // namespace

size_t attend_counter_bytes() { return (sizeof(int) * kAttendMaxCtas + 255) / 256 * 256; }
size_t attend_workspace_bytes() {
  return attend_counter_bytes() + sizeof(float) * 2 * kAttendMaxCtas * Shape<128>::kPart;
}

cudaError_t launch_attend(const AttendLaunch& in, cudaStream_t stream) {
  AttendLaunch L = in;
  L.ctas = kNumSMs * (L.a.dtype == PSPEC_BF16 ? 3 : 2);
  if (L.a.dtype == PSPEC_BF16)
    return L.a.D == 64 ? launch_d<64, BF16Tag>(L, stream) : launch_d<128, BF16Tag>(L, stream);
  return L.a.D == 64 ? launch_d<64, F32Tag>(L, stream) : launch_d<128, F32Tag>(L, stream);
}

}  // namespace pspec
