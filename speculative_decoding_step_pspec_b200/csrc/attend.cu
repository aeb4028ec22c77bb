// attend.cu -- attention of a ragged batch over the 4-bit paged cache (one launch).
//
// Work: a tile is 8, 16 or 32 query rows (token x head of the group) of one sequence and kv head;
// its keys are cut into units of 64.  All units of all tiles form one list, dealt out evenly
// to persistent CTAs, so ragged lengths cost no balance and neither grid nor workspace depends
// on them.  A CTA's share covers at most two tiles partly (its first and its last); those go to
// the workspace as (max, sum, unnormalised output), and the CTA that arrives last joins them
// in key order.
//
// Per unit each of the four warps takes 16 keys and keeps its own running maximum and sum, so
// the loop has no barrier.  The cache's bytes come by asynchronous copies into a ring of the
// warp's own.  What costs is turning codes into fp16 (two conversions, two products and two
// shuffles of bits for every four values), so the cache is the wide operand of the tensor-core
// products -- 16 keys, or 16 of the values' columns, against 8 query rows -- and a converted
// fragment serves every group of 8 rows in the tile; few rows waste half as much as with the
// rows as the wide operand.  A dot product may run over the head dimension in any order, and a
// sum over keys in any order of keys, so the fragments are laid to the cache's bytes: a lane's
// 16 (or 8) bytes of one key ARE its fragments of 8 (or 4) products, and two keys' nibbles
// interleaved are the pairs that the product with the values wants.  Dequantised values are
// exact in fp16: 2 significant bits of the code times 4 of the scale, between 2^-10 and 2688.
//
// Probabilities go into the product as fp16: of 2^15 at most and 2^7 at a row's maximum, a bf16 row's
// are rounded to 11 bits, an eighth of what its output is rounded by (they are summed as they are); an
// fp32 row's, and its queries, are two such terms.  Its outputs are summed outside the products.
//
// Measured: one token of each of 64 sequences (540 thousand keys in all, 32 heads on 8, D = 128):
// 181 us, 3.27 TB/s or half of the measured copy bandwidth (fp32: 269 us); the conversions hold the
// integer pipe at 55 percent and issue at 61, with three CTAs an SM (four: 188 us, five: 202, both for
// want of registers), 18 percent of the warps.  One token over 100000 keys: 53 us, 33 of them at
// that rate, the rest starting and joining the 55 parts of a tile.  Tiles of 8 rows spill nothing (fp32:
// 8 bytes); bf16 tiles of 16 rows up to 208 bytes, of 32 rows up to 380.
#include "attend_common.cuh"

namespace pspec {

using namespace attention;

namespace {

constexpr int kAttWarps = 4;
constexpr int kAttThreads = 32 * kAttWarps;
constexpr int kStep = 16;                       // keys of one warp step
static_assert(kUnit == kStep * kAttWarps, "a step of each warp");
constexpr int kStages = 4;
constexpr int kAttendMaxCtas = kNumSMs * 4;
// Taken from the exponents of a row without a key yet: the lowest value, so that any score above it
// passes the slack and becomes the row's maximum.
constexpr float kNoMax = -3.402823466e38f;
// Persistent CTAs that fit an SM by their registers.
constexpr int attend_ctas_per_sm(int D, bool f32, int NT) {
  return NT == 1 ? (D == 64 ? 4 : 3) : (D == 64 && NT == 2 && !f32 ? 4 : (f32 ? 2 : 3));
}

template <int D, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;          // rows of a tile
  static constexpr int kLane = D / 4;           // values of a key that a lane holds
  static constexpr int kWords = D / 32;         // their 32-bit words
  static constexpr int kK = D / 16;             // products over the head dimension
  static constexpr int kM = D / 16;             // products over the output's columns
  static constexpr int kCols = D / 8;           // output columns that a lane holds, contiguous
  static constexpr int kRow = D / 2;            // bytes of a key
  static constexpr int kScaleRow = D / 16;
  static constexpr int kStage = 2 * kStep * (kRow + kScaleRow);
  static constexpr int kRing = kStages * kStage;
  static constexpr long long kPart = kRows * (D + 2);   // floats of a partial tile
};
constexpr long long kMaxPart = 32 * (64 + 2) > 16 * (128 + 2) ? 32 * (64 + 2) : 16 * (128 + 2);

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

// Transposes an 8 x 8 matrix of 16-bit elements, two of a row in each lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

template <int D, int NT>
struct AttendSmem {
  union {
    alignas(128) uint8_t ring[kAttWarps][Shape<D, NT>::kRing];
    float out[kAttWarps][Shape<D, NT>::kRows][D + 4];
  };
  float m[kAttWarps][Shape<D, NT>::kRows];
  float l[kAttWarps][Shape<D, NT>::kRows];
  unsigned live[kAttWarps][kStages];          // which of the stage's keys exist
  ShareSmem share;
  int last;
};

template <int D, typename Tag, bool kWholePages, int NT>
__global__ void __launch_bounds__(kAttThreads, attend_ctas_per_sm(D, sizeof(typename Tag::elem) == 4, NT))
attend_kernel(const AttendLaunch L) {
  using elem = typename Tag::elem;
  using S = Shape<D, NT>;
  constexpr int kTileRows = S::kRows;
  constexpr bool kF32 = sizeof(elem) == 4;     // two fp16 terms for queries and probabilities
  extern __shared__ __align__(128) uint8_t s_raw[];
  auto& sm = *reinterpret_cast<AttendSmem<D, NT>*>(s_raw);
  const pspec_attend_args& a = L.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int group = a.Hq / a.Hkv;
  const int cta = blockIdx.x;

  Share share;
  if (!share_of<kTileRows, kAttThreads>(a, group, L.ctas, sm.share, share)) return;
  const long long U = share.U, E = share.E, w1 = share.w1;
  int seq = share.seq;
  long long prefix = share.prefix;

  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm.ring[warp]);
  const uint8_t* ring_p = sm.ring[warp];
  // Row r of a product's 16 keys is key r/2 (r even) or 7 - r/2 (odd) of the lower or upper
  // eight, so that the keys of a lane's value pairs are t, 7-t, 8+t and 15-t; 16-byte chunks of
  // odd key pairs are swapped by two (D = 128) to keep the reads free of conflicts.
  const int tau = (g & 1) ? 7 - (g >> 1) : g >> 1;
  constexpr int kWalks = kWholePages ? 1 : (D == 128 ? 3 : 2);
  const int walk_key[3] = {kWholePages ? 0 : (D == 128 ? lane >> 2 : lane >> 1),
                           D == 128 ? (lane >> 2) + 8 : lane & 15, lane & 15};

  const int unit_cols = kUnit / a.block_size, unit_rest = kUnit - unit_cols * a.block_size;

  long long w = share.w0;
  bool first = true;
  Seq s = seq_of<kTileRows>(a, seq, group);
  while (w < w1) {
    while (w >= prefix + s.units * s.tiles * a.Hkv) {
      prefix += s.units * s.tiles * a.Hkv;
      s = seq_of<kTileRows>(a, ++seq, group);
    }
    const long long item = (w - prefix) / s.units;
    const long long item0 = prefix + item * s.units;          // the tile's first unit
    const int h = (int)(item / s.tiles);
    const long long r0 = (item - (long long)h * s.tiles) * kTileRows;
    const long long u0 = w - item0;
    const long long u1 = min(s.units, w1 - item0);
    w = item0 + u1;

    // the keys that the tile's rows may see: lane r < kTileRows looks at row r
    const RowRef rr = row_of(a, s, group, h, lane < kTileRows ? r0 + lane : (long long)s.rows * group);
    int lim_hi = rr.limit, lim_lo = rr.limit < 0 ? 0x7fffffff : rr.limit;
    lim_hi = __reduce_max_sync(0xffffffffu, lim_hi);
    lim_lo = __reduce_min_sync(0xffffffffu, lim_lo);
    const int* table = a.block_table + (long long)seq * a.max_blocks;
    const int steps = (int)(min(u1, ((long long)max(lim_hi, 0) + kUnit - 1) / kUnit) - u0);

    // ---- one step's copies, the pages looked up a step ahead
    const long long key0 = u0 * kUnit + warp * kStep;         // of step 0
    Walk walk[kWalks];
    int blk[kWalks];
    auto look = [&](int step) {
#pragma unroll
      for (int i = 0; i < kWalks; ++i)
        blk[i] = key0 + (long long)step * kUnit + walk_key[i] < s.len ? __ldg(table + walk[i].col) : -1;
    };
#pragma unroll
    for (int i = 0; i < kWalks; ++i) walk[i].set(key0 + walk_key[i], a.block_size);
    look(0);
    auto issue = [&](int step) {
      const int left = (int)max(0LL, min((long long)kStep, (long long)s.len - key0 - (long long)step * kUnit));
      const uint32_t dst = ring + (step % kStages) * S::kStage;
      long long row[kWalks];
      bool live[kWalks];
#pragma unroll
      for (int i = 0; i < kWalks; ++i) {
        live[i] = (unsigned)blk[i] < (unsigned)a.num_blocks;
        row[i] = live[i] ? ((long long)blk[i] * a.Hkv + h) * a.block_size + walk[i].off : 0;
        walk[i].advance(unit_cols, unit_rest, a.block_size);
      }
      look(step + 1);
      auto copies = [&](int key, int c, long long r, bool ok) {
        const long long at = r * S::kRow + c * 16;
        const uint32_t to = dst + key * S::kRow + (D == 128 ? (c ^ ((key >> 1 & 1) << 1)) << 4 : c << 4);
        cp_async16(to, static_cast<const uint8_t*>(a.k_pages) + at, ok);
        cp_async16(to + kStep * S::kRow, static_cast<const uint8_t*>(a.v_pages) + at, ok);
      };
      const int skey = lane & 15;
      bool ok;
      long long srow;
      if constexpr (kWholePages) {
        if constexpr (D == 128) {
          const int key = lane >> 2;
          copies(key, lane & 3, live[0] && key < left ? row[0] + key : 0, live[0] && key < left);
          copies(key + 8, lane & 3, live[0] && key + 8 < left ? row[0] + key + 8 : 0, live[0] && key + 8 < left);
        } else {
          const int key = lane >> 1;
          copies(key, lane & 1, live[0] && key < left ? row[0] + key : 0, live[0] && key < left);
        }
        ok = live[0] && skey < left;
        srow = ok ? row[0] + skey : 0;
      } else {
        if constexpr (D == 128) {
          copies(lane >> 2, lane & 3, row[0], live[0]);
          copies((lane >> 2) + 8, lane & 3, row[1], live[1]);
        } else {
          copies(lane >> 1, lane & 1, row[0], live[0]);
        }
        ok = live[kWalks - 1];
        srow = row[kWalks - 1];
      }
      const uint8_t* src = static_cast<const uint8_t*>(lane < 16 ? a.k_block_scales : a.v_block_scales) + srow * S::kScaleRow;
      cp_async_small<S::kScaleRow>(dst + 2 * kStep * S::kRow + lane * S::kScaleRow, src, ok);
      const unsigned alive = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      if (lane == 0) {
        sm.live[warp][step % kStages] = alive;
        // a key that exists but whose page does not is hidden
        if (alive != (1u << left) - 1u) set_err(a.err, PSPEC_DEVERR_BLOCK_RANGE);
      }
    };
    auto issue_next = [&](int step) {
      if (step < steps) issue(step);
      asm volatile("cp.async.commit_group;");
    };
    for (int st = 0; st < kStages - 1; ++st) issue_next(st);

    // ---- the query rows as fragments: lane (g, t) has a quarter of row 8n + g, power-of-two
    // scaled into fp16's range
    uint32_t qb[NT][S::kK][2], ql[kF32 ? NT : 1][S::kK][2];
    float mult[NT][2];                          // of rows 8n + 2t and 8n + 2t + 1
    int limit[NT][2];
    {
      const float ks = a.k_scale ? __ldg(a.k_scale + h) : 1.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const RowRef rq = row_of(a, s, group, h, r0 + 8 * n + g);
        float x[S::kLane];
        float top = 0.f;
        const long long tok = rq.at / a.Hq;
        const elem* p = static_cast<const elem*>(a.q) + tok * a.q_stride + (rq.at - tok * a.Hq) * D + t * S::kLane;
#pragma unroll
        for (int j = 0; j < S::kLane; j += 2) {
          x[j] = x[j + 1] = 0.f;
          if (rq.limit > 0) load_q2(p + j, x[j], x[j + 1]);
          top = fmaxf(top, fmaxf(fabsf(x[j]), fabsf(x[j + 1])));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^(14 - exponent of the row's largest element), kept within fp32's normal range
        const int ex = (int)(__float_as_uint(top) >> 23) - 127;
        const int up = top == 0.f || ex == 128 ? 0 : min(126, 14 - ex);
        const float f = __uint_as_float((unsigned)(127 + up) << 23);
        const float back = score_factor(a.scale, ks, up);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mult[n][r] = __shfl_sync(0xffffffffu, back, (2 * t + r) * 4);
          limit[n][r] = __shfl_sync(0xffffffffu, rq.limit, (2 * t + r) * 4);
        }
#pragma unroll
        for (int k = 0; k < S::kK; ++k)
#pragma unroll
          for (int pair = 0; pair < 2; ++pair) {
            const float u = x[4 * k + 2 * pair] * f, v = x[4 * k + 2 * pair + 1] * f;
            const uint32_t hi = pack_half(u, v);
            qb[n][k][pair] = hi;
            if constexpr (kF32) ql[n][k][pair] = pack_half(u - half_lo(hi), v - half_hi(hi));
          }
      }
    }

    // o[n][m]: rows 8n + 2t (elements 0, 2) and 8n + 2t + 1 (1, 3), columns kCols g + 2m, + 1
    float o[NT][S::kM][4];
    float m[NT][2], at[NT][2], l[NT][2];        // at: what is taken from the exponents
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < S::kM; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[n][j][c] = 0.f;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        m[n][r] = -INFINITY;
        at[n][r] = kNoMax;
        l[n][r] = 0.f;
      }
    }

    bool coarse = false;                        // some row's maximum is beyond kCoarse
    for (int step = 0; step < steps; ++step) {
      issue_next(step + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1));
      __syncwarp();
      const uint8_t* buf = ring_p + (step % kStages) * S::kStage;
      const long long k0 = (u0 + step) * kUnit + warp * kStep;
      const unsigned alive = sm.live[warp][step % kStages];

      // ---- scores: 16 keys x 8 NT rows
      float sc[NT][4] = {};
      {
        uint32_t wd[2][S::kWords], f[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int key = 8 * j + tau;
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(buf + key * S::kRow + ((t ^ ((key >> 1 & 1) << 1)) << 4));
            wd[j][0] = v.x; wd[j][1] = v.y; wd[j][2] = v.z; wd[j][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(buf + key * S::kRow + t * 8);
            wd[j][0] = v.x; wd[j][1] = v.y;
          }
          const uint8_t* sp = buf + 2 * kStep * S::kRow + key * S::kScaleRow;
          if constexpr (D == 128) {
            const uint32_t two = scales_to_half(*reinterpret_cast<const uint16_t*>(sp + 2 * t));
            f[j][0] = __byte_perm(two, 0, 0x1010);
            f[j][1] = __byte_perm(two, 0, 0x3232);
          } else {
            const uint32_t one = sp[t];
            f[j][0] = f[j][1] = scales_to_half(one | one << 8);
          }
        }
#pragma unroll
        for (int k = 0; k < S::kWords; ++k) {
          uint32_t x[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            codes_to_half(wd[j][k], x[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[j][i] = hmul2(x[j][i], f[j][2 * k < S::kWords ? 0 : 1]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t fr[4] = {x[0][2 * i], x[1][2 * i], x[0][2 * i + 1], x[1][2 * i + 1]};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(sc[n], fr, qb[n][2 * k + i][0], qb[n][2 * k + i][1]);
              if constexpr (kF32) mma16816(sc[n], fr, ql[n][2 * k + i][0], ql[n][2 * k + i][1]);
            }
          }
        }
      }

      // ---- softmax in base 2: exponents less what each row takes; the maximum is looked for only
      // when one of them passes the slack
      const bool masked = alive != 0xffffu || k0 + kStep > lim_lo;
      auto exponents = [&](float (&y)[NT][4], bool rounded) {
        if (rounded) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) y[n][c] = __fadd_rn(__fmul_rn(sc[n][c], mult[n][c & 1]), -at[n][c & 1]);
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) y[n][c] = fmaf(sc[n][c], mult[n][c & 1], -at[n][c & 1]);
        }
        if (masked) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int key = (c & 2 ? 8 : 0) + tau;
              if (!(alive >> key & 1) || k0 + key >= limit[n][c & 1]) y[n][c] = -INFINITY;
            }
        }
      };
      float y[NT][4];
      exponents(y, false);
      bool grow = coarse;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) grow |= y[n][c] > kShift + kSlack;
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float top = -INFINITY;
            if (y[n][r] > -INFINITY) top = __fmul_rn(sc[n][r], mult[n][r]);
            if (y[n][r + 2] > -INFINITY) top = fmaxf(top, __fmul_rn(sc[n][r + 2], mult[n][r]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float old = m[n][r];
            m[n][r] = fmaxf(old, top);
            if (m[n][r] > old) {
              const float f = ex2(old - m[n][r]);
              at[n][r] = m[n][r] - kShift;
              coarse |= fabsf(m[n][r]) >= kCoarse;
              l[n][r] *= f;
#pragma unroll
              for (int j = 0; j < S::kM; ++j) {
                o[n][j][r] *= f;
                o[n][j][r + 2] *= f;
              }
            }
          }
        coarse = __any_sync(0xffffffffu, coarse);
        exponents(y, coarse);
      }
      uint32_t pb[NT][2], pl[kF32 ? NT : 1][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float u = ex2(y[n][2 * j]), v = ex2(y[n][2 * j + 1]);
          l[n][0] += u;
          l[n][1] += v;
          const uint32_t hi = pack_half(u, v);
          pb[n][j] = transpose8(hi);
          if constexpr (kF32) pl[n][j] = transpose8(pack_half(u - half_lo(hi), v - half_hi(hi)));
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
        uint32_t fr[4][4];                                  // of 4 products: even, odd columns of
#pragma unroll                                              // the first pair of keys, of the second
        for (int pr = 0; pr < 2; ++pr)
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const uint32_t x = vw[2 * pr][k], y = vw[2 * pr + 1][k];
            const uint32_t both = odd ? ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u)
                                      : (x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u);
            uint32_t b[4];
            codes_to_half(both, b);
#pragma unroll
            for (int i = 0; i < 4; ++i) fr[i][2 * pr + odd] = hmul2(b[i], f[pr]);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if constexpr (kF32) {
              // the step's sum by itself: the tensor cores cut a sum's last bits off, which along
              // thousands of keys adds up (17792 keys: outputs off by 8e-6, added like this by 1e-6)
              float x[4] = {};
              mma16816(x, fr[i], pl[n][0], pl[n][1]);
              mma16816(x, fr[i], pb[n][0], pb[n][1]);
#pragma unroll
              for (int c = 0; c < 4; ++c) o[n][4 * k + i][c] += x[c];
            } else {
              mma16816(o[n][4 * k + i], fr[i], pb[n][0], pb[n][1]);
            }
          }
      }
      __syncwarp();                                         // the stage may be refilled
    }
    asm volatile("cp.async.wait_group 0;");
    __syncthreads();                                        // every warp is done with its ring

    // ---- the four warps' results joined
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], x);
        const int row = 8 * n + 2 * t + r;
        if (g == 0) {
          sm.m[warp][row] = m[n][r];
          sm.l[warp][row] = l[n][r];
        }
#pragma unroll
        for (int j = 0; j < S::kM; j += 2)
          *reinterpret_cast<float4*>(&sm.out[warp][row][S::kCols * g + 2 * j]) =
              make_float4(o[n][j][r], o[n][j][r + 2], o[n][j + 1][r], o[n][j + 1][r + 2]);
      }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == s.units;
    float* part = L.parts + (2LL * cta + (first ? 0 : 1)) * S::kPart;
    first = false;
    const float vscale = a.v_scale ? __ldg(a.v_scale + h) : 1.f;
    auto finish = [&](const RowRef& rr, int d, float M, float sum, float4 v) {
      finish_row<D, elem>(a, rr, d, M, sum, vscale, v);
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
        auto part_of = [&](long long c) { return L.parts + (c == cta_a ? slot_a : 2 * c) * S::kPart; };
        const int n = (int)(cta_b - cta_a) + 1;
        constexpr int kSeats = kAttThreads / kTileRows;     // threads of a row
        constexpr int kBatch = 32;                          // parts whose factors are held at once
        constexpr int kHeld = kTileRows * (D / 4) / kAttThreads;
        float* seat = reinterpret_cast<float*>(s_raw);      // [kSeats][rows], then [rows]
        float* factor = seat + kAttThreads + kTileRows;     // [kBatch][rows]
        const int row = tid % kTileRows, place = tid / kTileRows;
        float M = -INFINITY;
#pragma unroll 4
        for (int c = place; c < n; c += kSeats) M = fmaxf(M, ld_cg(part_of(cta_a + c) + kTileRows * D + row));
        seat[tid] = M;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSeats; ++i) M = fmaxf(M, seat[i * kTileRows + row]);
        float sum = 0.f;
        float4 v[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = 0; c0 < n; c0 += kBatch) {
          const int nb = min(kBatch, n - c0);
          __syncthreads();
#pragma unroll 4
          for (int c = place; c < nb; c += kSeats) {
            const float* p = part_of(cta_a + c0 + c) + kTileRows * D + row;
            const float mc = ld_cg(p), lc = ld_cg(p + kTileRows);
            const float f = mc == -INFINITY ? 0.f : ex2(mc - M);
            factor[c * kTileRows + row] = f;
            sum += f * lc;
          }
          __syncthreads();
          constexpr int kParts = 16 / kHeld;                // sixteen loads in flight
          for (int c1 = 0; c1 < nb; c1 += kParts) {
            float4 x[kParts][kHeld];
#pragma unroll
            for (int c = 0; c < kParts; ++c)
#pragma unroll
              for (int i = 0; i < kHeld; ++i)
                x[c][i] = ld_cg(reinterpret_cast<const float4*>(part_of(cta_a + c0 + min(c1 + c, nb - 1))) + i * kAttThreads + tid);
#pragma unroll
            for (int c = 0; c < kParts; ++c)
#pragma unroll
              for (int i = 0; i < kHeld; ++i) {
                const float f = c1 + c < nb ? factor[(c1 + c) * kTileRows + (i * kAttThreads + tid) / (D / 4)] : 0.f;
                if (f != 0.f) {                             // (a part without a key may hold anything)
                  v[i].x += f * x[c][i].x; v[i].y += f * x[c][i].y; v[i].z += f * x[c][i].z; v[i].w += f * x[c][i].w;
                }
              }
          }
        }
        __syncthreads();
        seat[tid] = sum;
        if (place == 0) factor[row] = M;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          const int at = i * kAttThreads + tid, r = at / (D / 4);
          float total = 0.f;
#pragma unroll
          for (int x = 0; x < kSeats; ++x) total += seat[x * kTileRows + r];
          finish(row_of(a, s, group, h, r0 + r), (at - r * (D / 4)) * 4, factor[r], total, v[i]);
        }
      }
    }
    __syncthreads();                                        // shared memory is the ring's again
  }
}

template <int D, typename Tag, int NT>
cudaError_t launch_nt(AttendLaunch L, cudaStream_t stream) {
  constexpr int smem = sizeof(AttendSmem<D, NT>);
  constexpr int ctas = attend_ctas_per_sm(D, sizeof(typename Tag::elem) == 4, NT);
  static_assert(smem <= 48 * 1024 && smem * ctas <= 220 * 1024, "within the default limit, and all fit");
  static_assert(Shape<D, NT>::kPart <= kMaxPart && ctas * kNumSMs <= kAttendMaxCtas, "within the workspace");
  L.ctas = kNumSMs * ctas;
  auto* fn = L.a.block_size % kStep == 0 ? attend_kernel<D, Tag, true, NT> : attend_kernel<D, Tag, false, NT>;
  fn<<<L.ctas, kAttThreads, smem, stream>>>(L);
  return cudaGetLastError();
}

// The largest tiles of which there are three to an SM (about the CTAs that fit): fewer leave each to
// many CTAs, whose results take longer to join than a code takes to be converted again (8 rows of 64
// heads over 4096 keys: 23 us in tiles of 8 rows, 43 in tiles of 32).
template <int D, typename Tag>
cudaError_t launch_d(const AttendLaunch& L, cudaStream_t stream) {
  const long long rows = ((long long)L.a.T * (L.a.Hq / L.a.Hkv) + L.a.B - 1) / L.a.B;
  constexpr int most = D == 64 && sizeof(typename Tag::elem) == 2 ? 4 : 2;
  const auto fits = [&](int nt) {
    return rows > 4 * nt && (long long)L.a.B * L.a.Hkv * ((rows + 8 * nt - 1) / (8 * nt)) >= 3 * kNumSMs;
  };
  if (most == 4 && fits(4)) return launch_nt<D, Tag, most>(L, stream);
  if (fits(2)) return launch_nt<D, Tag, 2>(L, stream);
  return launch_nt<D, Tag, 1>(L, stream);
}

}  // namespace

size_t attend_counter_bytes() {
  static_assert(sizeof(int) * kAttendMaxCtas <= PSPEC_ATTEND_ZERO_BYTES, "all counters");
  return PSPEC_ATTEND_ZERO_BYTES;
}
size_t attend_workspace_bytes() {
  const size_t parts = sizeof(float) * 2 * kAttendMaxCtas * kMaxPart, wide = attend_wide_part_bytes();
  return (attend_counter_bytes() + (parts > wide ? parts : wide) + 255) / 256 * 256;
}

cudaError_t launch_attend(const AttendLaunch& L, cudaStream_t stream) {
  if (attend_is_wide(L)) return launch_attend_wide(L, stream);
  if (L.a.dtype == PSPEC_BF16)
    return L.a.D == 64 ? launch_d<64, BF16Tag>(L, stream) : launch_d<128, BF16Tag>(L, stream);
  return L.a.D == 64 ? launch_d<64, F32Tag>(L, stream) : launch_d<128, F32Tag>(L, stream);
}

}  // namespace pspec
