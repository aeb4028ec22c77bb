// attend_wide.cu -- attention over the 4-bit paged cache for many query rows (one launch).
//
// The same list of work as attend.cu's with tiles of 128 rows: a sequence's rows share a kv head's
// keys, so each key is converted to fp16 once for 128 rows, and both products run on the fifth
// generation's tensor cores with their sums in tensor memory.  Two CTAs to an SM, each
//   8 warps of softmax, two threads to a row: the scores of 64 keys come out of tensor memory,
//     become probabilities in registers and go back over them as fp16; the two threads of a row
//     agree on its maximum, which moves rarely;
//   4 warps each for the keys and the values: codes are fetched some units ahead, converted and
//     laid into shared memory as the 128-byte swizzled tiles that the products read, two buffers
//     each;
//   1 warp that issues the products: scores of units n + 1 and n + 2 are on their way while the
//     softmax has unit n.
// A unit of 64 keys is 64 x 128 exponentials; 16 a clock bound a full tile's unit at 512 clocks of
// an SM, its products (D = 64) at 256.  Latency is what costs: with half the warps for each role
// a unit took 2350 clocks of a CTA, the instructions of each one after another.  Warps without a
// live row skip theirs.
//
// Measured: 64 draft batches (1 to 15 rows of 64 heads on 8 each, D = 64): 361 us, 164 TFLOP/s;
// prompts of 200 to 700 rows (16 heads on 2, D = 128): 161 us, 220 TFLOP/s.  Latency bounds it: a unit
// takes 2640 warp instructions before a second warp of softmax has live rows, most of them in the
// conversions and around them, which fill 61 (44) percent of the active issue slots with 48 percent of
// the warps; the tensor cores are busy for 20 (14).  Among what is waited for are spilled registers:
// 56 for every role, 348 bytes of spills for D = 64, 572 for D = 128.
//
// Probabilities are rounded to fp16 on their way into the product (11 bits, an eighth of the output's
// rounding to bf16) and summed as they are.
//
// Every wait has a limit, after which the CTA goes on without waiting, sets PSPEC_DEVERR_WAIT and
// ends as usual.
#include "attend_common.cuh"

namespace pspec {

using namespace attention;

namespace {

constexpr int kWideRows = 128;
constexpr int kSoftThreads = 256, kFillThreads = 128;     // fillers: of keys, and of values
constexpr int kWideThreads = kSoftThreads + 2 * kFillThreads + 32;
constexpr int kJoinThreads = 256;               // that join a tile's parts
constexpr int kWideCtas = 2 * kNumSMs;
constexpr uint32_t kTmemCols = 256;             // scores in two buffers of 64, outputs
constexpr uint32_t kTmemOut = 128;
constexpr long long kWaitClocks = 1ll << 31;     // about a second
constexpr int kBatch = 32;                      // parts whose factors are held at once

template <int D>
struct Wide {
  static constexpr int kPanels = D / 64;        // tiles are panels of 64 elements, 128 bytes a row
  static constexpr int kQ = kPanels * kWideRows * 128;
  static constexpr int kTile = kPanels * kUnit * 128;
  static constexpr int kRow = D / 2;            // bytes of a key in the cache
  static constexpr int kScaleRow = D / 16;
  static constexpr int kChunks = D / 64;        // 16-byte pieces of a key's codes per thread
  static constexpr int kLanes = D / 32;         // threads of a key
  static constexpr int kStep = kFillThreads / kLanes;   // keys of one piece
  static constexpr int kAhead = D == 64 ? 2 : 1;        // units fetched ahead
  static constexpr long long kPart = kWideRows * (D + 2);
};

template <int D>
struct WideSmem {
  union {
    uint8_t q[Wide<D>::kQ];
    float factor[kBatch * kWideRows];
  };
  uint8_t k[2][Wide<D>::kTile];
  uint8_t v[2][Wide<D>::kTile];
  unsigned long long k_full[2], v_full[2], s_full[2], p_full[2], pv_done[2];
  // of four units, for their keys may be laid before the softmax of the second last has read them
  alignas(8) uint8_t live[4][kUnit];            // which of the keys exist
  int dead[4];                                  // the last unit here with one that does not
  float seat[kJoinThreads];
  float top[kWideRows];
  int hi[4], lo[4];
  uint32_t tmem;
  int failed, last;
  ShareSmem share;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(unsigned long long* b, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t a) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(a) : "memory");
}
__device__ __forceinline__ bool bar_done(uint32_t a, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(done) : "r"(a), "r"(parity) : "memory");
  return done != 0;
}
__device__ __noinline__ void bar_wait_long(uint32_t a, uint32_t parity, volatile int* failed) {
  const long long start = clock64();
  while (!bar_done(a, parity)) {
    if (*failed) return;
    if (clock64() - start > kWaitClocks) *failed = 1;
  }
}
__device__ __forceinline__ void bar_wait(uint32_t a, uint32_t parity, volatile int* failed) {
#pragma unroll 1
  for (int i = 0; i < 8; ++i)
    if (bar_done(a, parity)) return;
  bar_wait_long(a, parity, failed);
}
__device__ __forceinline__ void bar_wait(unsigned long long* b, uint32_t parity, volatile int* failed) {
  bar_wait(smem_addr(b), parity, failed);
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(unsigned long long* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(b)) : "memory");
}

// A tile's descriptor: 128-byte swizzle, rows of 128 bytes in groups of eight 1024 bytes apart;
// `panel`: bytes between panels of 64 elements, for an operand that is read along them.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t panel) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(panel >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// fp16 operands, fp32 sums, 128 rows x N columns; transposed: B is read along its rows.
__host__ __device__ constexpr uint32_t product_kind(int N, bool transposed) {
  return 1u << 4 | (transposed ? 1u << 16 : 0u) | (uint32_t)(N / 8) << 17 | (128u / 16) << 24;
}
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               ::"r"(d), "l"(a), "l"(b), "r"(kind), "r"((int)add) : "memory");
}
__device__ __forceinline__ void product_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
               ::"r"(d), "r"(a), "l"(b), "r"(kind), "r"((int)add) : "memory");
}

// 16 columns of the lane's row.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&x)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]),
                 "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&x)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
               ::"r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]),
                 "r"(x[8]), "r"(x[9]), "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]),
                 "r"(addr) : "memory");
}
// (x passes through, so that nothing is done with it before)
__device__ __forceinline__ void tmem_wait_load(uint32_t (&x)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                 "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15])
               ::"memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The two warps that share 32 rows: meet, and whether a lane of either says so.
__device__ __forceinline__ bool pair_any(int pair, bool x) {
  int r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.aligned.pred q, %2, 64, p;\n\t"
               "selp.b32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"((int)x), "r"(pair + 1) : "memory");
  return r != 0;
}
__device__ __forceinline__ bool elected() {
  int r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Byte offset of 16-byte chunk c of row r in a swizzled panel.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// 32 codes (a key's 16-byte piece) with their two block scales as fp16 into four chunks of a
// tile's row, the first at shared address `at`: chunk i lies 16 i away but for the swizzle.
__device__ __forceinline__ void convert(uint32_t at, const uint4& codes, uint32_t scales) {
  const uint32_t two = scales_to_half(scales);
  const uint32_t f[2] = {__byte_perm(two, 0, 0x1010), __byte_perm(two, 0, 0x3232)};
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[4];
    codes_to_half(w[i], h);
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (16u * i)), "r"(hmul2(h[0], f[i >> 1])),
                 "r"(hmul2(h[1], f[i >> 1])), "r"(hmul2(h[2], f[i >> 1])), "r"(hmul2(h[3], f[i >> 1])) : "memory");
  }
}

template <int D>
__global__ void __launch_bounds__(kWideThreads, 2) attend_wide_kernel(const AttendLaunch L) {
  using S = Wide<D>;
  extern __shared__ uint8_t s_raw[];
  auto& sm = *reinterpret_cast<WideSmem<D>*>(s_raw + ((1024 - (smem_addr(s_raw) & 1023)) & 1023));
  const pspec_attend_args& a = L.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = a.Hq / a.Hkv;
  const int cta = blockIdx.x;

  Share share;
  if (!share_of<kWideRows, kWideThreads>(a, group, L.ctas, sm.share, share)) return;
  const long long U = share.U, E = share.E, w1 = share.w1;
  int seq = share.seq;
  long long prefix = share.prefix;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      bar_init(&sm.k_full[b], kFillThreads);
      bar_init(&sm.v_full[b], kFillThreads);
      bar_init(&sm.s_full[b], 1);
      bar_init(&sm.p_full[b], kSoftThreads);
      bar_init(&sm.pv_done[b], 1);
      sm.dead[b] = sm.dead[b + 2] = -1;
    }
    sm.failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sm.tmem;
  volatile int* failed = &sm.failed;

  int base = 0;                                 // units that the CTA has done: buffers and phases
  long long w = share.w0;
  bool first = true;
  Seq s = seq_of<kWideRows>(a, seq, group);
  while (w < w1) {
    while (w >= prefix + s.units * s.tiles * a.Hkv) {
      prefix += s.units * s.tiles * a.Hkv;
      s = seq_of<kWideRows>(a, ++seq, group);
    }
    const long long item = (w - prefix) / s.units;
    const long long item0 = prefix + item * s.units;          // the tile's first unit
    const int h = (int)(item / s.tiles);
    const long long r0 = (item - (long long)h * s.tiles) * kWideRows;
    const long long u0 = w - item0;
    const long long u1 = min(s.units, w1 - item0);
    w = item0 + u1;

    // ---- the rows' limits, and the query rows as fp16, power-of-two scaled into its range
    const int row = tid & (kWideRows - 1), half = tid / kWideRows;   // (softmax threads)
    RowRef rr{0, -1};
    float mult = 0.f;
    if (warp < 8) {
      rr = row_of(a, s, group, h, r0 + row);
      const int hi = __reduce_max_sync(0xffffffffu, rr.limit);
      const int lo = __reduce_min_sync(0xffffffffu, rr.limit < 0 ? 0x7fffffff : rr.limit);
      if (lane == 0 && warp < 4) {
        sm.hi[warp] = hi;
        sm.lo[warp] = lo;
      }
      const long long tok = rr.at / a.Hq;
      const uint16_t* p = static_cast<const uint16_t*>(a.q) + tok * a.q_stride + (rr.at - tok * a.Hq) * D;
      const bool vec = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && a.q_stride % 8 == 0;
      auto load = [&](int c, float (&x)[8]) {
        if (rr.limit <= 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = 0.f;
        } else if (vec) {
          unpack(__ldg(reinterpret_cast<const uint4*>(p) + c), x, BF16Tag{});
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = load_scalar(p, 8 * c + i);
        }
      };
      float top = 0.f;
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        float x[8];
        load(c, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
      }
      // 2^(14 - exponent of the row's largest element), kept within fp32's normal range
      const int ex = (int)(__float_as_uint(top) >> 23) - 127;
      const int up = top == 0.f || ex == 128 ? 0 : min(126, 14 - ex);
      const float f = __uint_as_float((unsigned)(127 + up) << 23);
      mult = score_factor(a.scale, a.k_scale ? __ldg(a.k_scale + h) : 1.f, up);
#pragma unroll 2
      for (int c = half * (D / 16); c < (half + 1) * (D / 16); ++c) {
        float x[8];
        load(c, x);
        *reinterpret_cast<uint4*>(sm.q + (c >> 3) * (kWideRows * 128) + chunk_at(row, c & 7)) =
            make_uint4(pack_half(x[0] * f, x[1] * f), pack_half(x[2] * f, x[3] * f), pack_half(x[4] * f, x[5] * f), pack_half(x[6] * f, x[7] * f));
      }
      fence_async();
    }
    tc_before();
    __syncthreads();
    tc_after();
    const int lim_hi = max(max(sm.hi[0], sm.hi[1]), max(sm.hi[2], sm.hi[3]));
    const int steps = max(0, (int)(min(u1, ((long long)max(lim_hi, 0) + kUnit - 1) / kUnit) - u0));

    float m = -INFINITY, at = 0.f, l = 0.f;
    bool coarse = false;                                      // some row of the warp is beyond kCoarse
    if (warp < 8) {
      // ---- softmax
      const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21);   // the warp's 32 lanes
      const int warp_hi = sm.hi[warp & 3] < 0 ? -1 : (int)max(0LL, sm.hi[warp & 3] - u0 * kUnit);
      const int warp_lo = (int)max(0LL, sm.lo[warp & 3] - u0 * kUnit);
      const int limit = (int)max(0LL, rr.limit - u0 * kUnit);
      for (int step = 0; step < steps; ++step) {
        const int n = base + step, b = n & 1;
        const int k0 = step * kUnit;                          // (limits are counted from there too)
        const uint32_t sc = mine + b * 64 + half * 32;        // the thread's 32 keys
        bar_wait(&sm.s_full[b], (n >> 1) & 1, failed);
        __syncwarp();
        tc_after();
        if (k0 < warp_hi) {                                   // else no row sees the unit ...
          // some key is hidden from some row: which ones this row sees
          const bool masked = k0 + kUnit > warp_lo || sm.dead[n & 3] == n;
          uint32_t seen = 0;
          if (masked) {
            const int left = max(0, min(32, limit - k0 - half * 32));
#pragma unroll
            for (int i = 0; i < 4; ++i) {                     // a byte of 0 or 1 per key: eight to bits
              const unsigned long long x = *reinterpret_cast<const unsigned long long*>(&sm.live[n & 3][half * 32 + 8 * i]);
              seen |= (uint32_t)((x * 0x0102040810204080ull) >> 56) << (8 * i);
            }
            seen &= left == 0 ? 0u : 0xffffffffu >> (32 - left);
          }
          // probabilities by the maximum so far; where one passes the slack, once more by the new
          uint32_t p[16];
          float sum[2], top;
          auto pass = [&](bool rounded) {
            float tops[2] = {-INFINITY, -INFINITY};
            sum[0] = sum[1] = 0.f;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              uint32_t x[16];
              tmem_load(sc + 16 * part, x);
              tmem_wait_load(x);
              if (rounded) {
#pragma unroll
                for (int c = 0; c < 16; ++c) x[c] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(x[c]), mult), -at));
              } else {
#pragma unroll
                for (int c = 0; c < 16; ++c) x[c] = __float_as_uint(fmaf(__uint_as_float(x[c]), mult, -at));
              }
              if (masked) {
                const uint32_t bits = seen >> (16 * part);
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  if (!(bits >> c & 1)) x[c] = __float_as_uint(-INFINITY);
              }
#pragma unroll
              for (int c = 0; c < 16; c += 2) {
                const float y = __uint_as_float(x[c]), z = __uint_as_float(x[c + 1]);
                tops[c >> 1 & 1] = fmax3(tops[c >> 1 & 1], y, z);
                const float u = ex2(y), v = ex2(z);
                sum[c >> 1 & 1] += u + v;
                p[8 * part + (c >> 1)] = pack_half(u, v);
              }
            }
            top = fmaxf(tops[0], tops[1]);
          };
          pass(false);
          const float most = m == -INFINITY ? -INFINITY : kShift + kSlack;
          if (pair_any(warp & 3, top > most || coarse)) {
            sm.seat[tid] = top;
            pair_any(warp & 3, false);
            top = fmaxf(top, sm.seat[tid ^ kWideRows]);
            float f = 1.f, now = top + at;
            // (both warps of the pair see the same rows, so they agree)
            coarse = __any_sync(0xffffffffu, coarse || (top > most && fmaxf(fabsf(now), fabsf(at)) >= kCoarse));
            if (coarse) {                                     // the products themselves
              now = -INFINITY;
#pragma unroll 1
              for (int part = 0; part < 2; ++part) {
                uint32_t x[16];
                tmem_load(sc + 16 * part, x);
                tmem_wait_load(x);
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  if (!masked || (seen >> (16 * part + c) & 1)) now = fmaxf(now, __fmul_rn(__uint_as_float(x[c]), mult));
              }
              pair_any(warp & 3, false);
              sm.seat[tid] = now;
              pair_any(warp & 3, false);
              now = fmaxf(now, sm.seat[tid ^ kWideRows]);
              top = now - at;
            }
            if (top > most) {
              f = ex2(m - now);
              m = now;
              at = now - kShift;
              l *= f;
            }
            if (step > 0) {
              bar_wait(&sm.pv_done[b ^ 1], ((n - 1) >> 1) & 1, failed);
              __syncwarp();
              tc_after();
#pragma unroll 1
              for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
                uint32_t o[16];
                tmem_load(mine + kTmemOut + c, o);
                tmem_wait_load(o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_store(mine + kTmemOut + c, o);
              }
            }
            pass(coarse);
          }
          l += sum[0] + sum[1];
          tmem_store(sc, p);
          tmem_wait_store();
        } else if (warp_hi > 0) {                             // ... and the products get zeros
          const uint32_t z[16] = {};
          tmem_store(sc, z);
          tmem_wait_store();
        }
        tc_before();
        bar_arrive(smem_addr(&sm.p_full[b]));
      }
    } else if (warp < 16) {
      // ---- keys (four warps) and values (four) into shared memory
      const bool is_k = warp < 12;
      const int ft = tid & (kFillThreads - 1);
      const int c = ft % S::kLanes, key = ft / S::kLanes;     // the thread's piece of its keys
      const int* table = a.block_table + (long long)seq * a.max_blocks;
      const int unit_cols = kUnit / a.block_size, unit_rest = kUnit - unit_cols * a.block_size;
      const int left = (int)((long long)s.len - u0 * kUnit) - key;    // keys from the thread's first on
      const uint8_t* pages = static_cast<const uint8_t*>(is_k ? a.k_pages : a.v_pages) + c * 16;
      const uint8_t* scales = static_cast<const uint8_t*>(is_k ? a.k_block_scales : a.v_block_scales) + c * 2;
      const int page = a.Hkv * a.block_size, head = h * a.block_size;
      Walk walk[S::kChunks];
      int blk[S::kChunks], next = 0;                          // pages of unit `next`
      struct Codes {
        uint4 x[S::kChunks];
        uint32_t s[S::kChunks];
        uint32_t live;                                        // bit i: the key of piece i exists
      } codes[S::kAhead];
      auto look = [&]() {
#pragma unroll
        for (int i = 0; i < S::kChunks; ++i)
          blk[i] = next < steps && next * kUnit + i * S::kStep < left ? __ldg(table + walk[i].col) : -1;
      };
      // codes of the unit whose pages were looked up; the next unit's pages are looked up
      auto fetch = [&](Codes& x) {
        x.live = 0;
#pragma unroll
        for (int i = 0; i < S::kChunks; ++i) {
          x.x[i] = make_uint4(0, 0, 0, 0);
          x.s[i] = 0;
          if ((unsigned)blk[i] < (unsigned)a.num_blocks) {
            x.live |= 1u << i;
            const long long at = (long long)blk[i] * page + (head + walk[i].off);
            x.x[i] = ld_stream(pages + at * S::kRow);
            x.s[i] = __ldg(reinterpret_cast<const unsigned short*>(scales + at * S::kScaleRow));
          }
          walk[i].advance(unit_cols, unit_rest, a.block_size);
        }
        ++next;
        look();
      };
#pragma unroll
      for (int i = 0; i < S::kChunks; ++i) walk[i].set(u0 * kUnit + key + i * S::kStep, a.block_size);
      look();
#pragma unroll
      for (int j = 0; j < S::kAhead; ++j) fetch(codes[j]);
      const uint32_t free_bar = smem_addr(is_k ? sm.s_full : sm.pv_done), full_bar = smem_addr(is_k ? sm.k_full : sm.v_full);
      // the thread's first chunk; its other keys lie whole groups of eight rows further
      const uint32_t dst = smem_addr(is_k ? sm.k[0] : sm.v[0]) + (c >> 1) * (kUnit * 128) + chunk_at(key, (c & 1) * 4);
      for (int step0 = 0; step0 < steps; step0 += S::kAhead) {
#pragma unroll
        for (int j = 0; j < S::kAhead; ++j) {
          const int step = step0 + j;
          if (step >= steps) break;
          const int n = base + step, b = n & 1;
          if (n >= 2) bar_wait(free_bar + 8 * b, ((n >> 1) - 1) & 1, failed);   // the buffer's previous use
#pragma unroll
          for (int i = 0; i < S::kChunks; ++i) {
            convert(dst + b * S::kTile + i * (S::kStep * 128), codes[j].x[i], codes[j].s[i]);
            if (is_k && c == 0) {
              const bool live = codes[j].live >> i & 1;
              sm.live[n & 3][key + i * S::kStep] = live;
              if (!live) {
                sm.dead[n & 3] = n;
                // a key that exists but whose page does not is hidden
                if (step * kUnit + i * S::kStep < left) set_err(a.err, PSPEC_DEVERR_BLOCK_RANGE);
              }
            }
          }
          fence_async();
          bar_arrive(full_bar + 8 * b);
          fetch(codes[j]);
        }
      }
    } else if (steps > 0) {
      // ---- products, by one lane; the warp stays together
      const bool lead = elected();
      const uint64_t qd = tile_desc(smem_addr(sm.q), 16), kd = tile_desc(smem_addr(sm.k[0]), 16),
                     vd = tile_desc(smem_addr(sm.v[0]), kUnit * 128);
      auto scores = [&](int n) {
        const int b = n & 1;
        const uint64_t kb = kd + b * (S::kTile >> 4);
        bar_wait(&sm.k_full[b], (n >> 1) & 1, failed);
        __syncwarp();
        tc_after();
        if (lead) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            product(tmem + b * 64, qd + ((k >> 2) * (kWideRows * 128) + (k & 3) * 32 >> 4), kb + ((k >> 2) * (kUnit * 128) + (k & 3) * 32 >> 4),
                    product_kind(kUnit, false), k > 0);
          tc_commit(&sm.s_full[b]);
        }
        __syncwarp();
      };
      scores(base);
      if (steps > 1) scores(base + 1);
      for (int step = 0; step < steps; ++step) {
        const int n = base + step, b = n & 1;
        const uint32_t parity = (n >> 1) & 1;
        bar_wait(&sm.v_full[b], parity, failed);
        bar_wait(&sm.p_full[b], parity, failed);
        __syncwarp();
        tc_after();
        if (lead) {
#pragma unroll
          for (int k = 0; k < kUnit / 16; ++k)                // probabilities: 16 columns of each 32
            product_tmem(tmem + kTmemOut, tmem + b * 64 + (k >> 1) * 32 + (k & 1) * 8, vd + (b * S::kTile + k * 2048 >> 4),
                         product_kind(D, true), step > 0 || k > 0);
          tc_commit(&sm.pv_done[b]);
        }
        __syncwarp();
        if (step + 2 < steps) {
          bar_wait(&sm.pv_done[b], parity, failed);           // the probabilities have been read
          scores(n + 2);
        }
      }
    }
    __syncwarp();

    // ---- the tile's outputs
    const bool whole = u0 == 0 && u1 == s.units;
    float* part = L.parts + (2LL * cta + (first ? 0 : 1)) * S::kPart;
    first = false;
    const float vscale = a.v_scale ? __ldg(a.v_scale + h) : 1.f;
    if (warp < 8) {
      if (steps > 0) {
        const int n = base + steps - 1;
        bar_wait(&sm.pv_done[n & 1], (n >> 1) & 1, failed);
        __syncwarp();
        tc_after();
      }
      sm.seat[tid] = l;
      pair_any(warp & 3, false);
      l += sm.seat[tid ^ kWideRows];
#pragma unroll 1
      for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
        uint32_t o[16];
        tmem_load(tmem + ((uint32_t)(warp & 3) << 21) + kTmemOut + c, o);
        tmem_wait_load(o);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          // (without a key that it sees a row has no output in tensor memory)
          float4 v = make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
          if (m == -INFINITY && l == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (whole) finish_row<D, uint16_t>(a, rr, c + i, m, l, vscale, v);
          else *reinterpret_cast<float4*>(part + row * D + c + i) = v;
        }
      }
      if (!whole && half == 0) {
        part[kWideRows * D + row] = m;
        part[kWideRows * D + kWideRows + row] = l;
      }
    }
    base += steps;
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
        constexpr int kSeats = kJoinThreads / kWideRows, kHeld = kWideRows * (D / 4) / kJoinThreads;
        const bool joins = tid < kJoinThreads;
        const int place = tid / kWideRows;
        float M = -INFINITY, sum = 0.f;
        if (joins) {
#pragma unroll 4
          for (int c = place; c < n; c += kSeats) M = fmaxf(M, ld_cg(part_of(cta_a + c) + kWideRows * D + row));
          sm.seat[tid] = M;
        }
        __syncthreads();
        if (joins) {
#pragma unroll
          for (int i = 0; i < kSeats; ++i) M = fmaxf(M, sm.seat[i * kWideRows + row]);
        }
        float4 v[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = 0; c0 < n; c0 += kBatch) {
          const int nb = min(kBatch, n - c0);
          __syncthreads();
          if (joins) {
#pragma unroll 4
            for (int c = place; c < nb; c += kSeats) {
              const float* p = part_of(cta_a + c0 + c) + kWideRows * D + row;
              const float mc = ld_cg(p), lc = ld_cg(p + kWideRows);
              const float f = mc == -INFINITY ? 0.f : ex2(mc - M);
              sm.factor[c * kWideRows + row] = f;
              sum += f * lc;
            }
          }
          __syncthreads();
          if (joins) {
            for (int c = 0; c < nb; ++c) {
              const float4* src = reinterpret_cast<const float4*>(part_of(cta_a + c0 + c));
#pragma unroll
              for (int i = 0; i < kHeld; ++i) {
                const int x = i * kJoinThreads + tid;
                const float4 y = ld_cg(src + x);
                const float f = sm.factor[c * kWideRows + x / (D / 4)];
                v[i].x += f * y.x; v[i].y += f * y.y; v[i].z += f * y.z; v[i].w += f * y.w;
              }
            }
          }
        }
        __syncthreads();
        if (joins) {
          sm.seat[tid] = sum;
          if (place == 0) sm.top[row] = M;
        }
        __syncthreads();
        if (joins) {
#pragma unroll
          for (int i = 0; i < kHeld; ++i) {
            const int x = i * kJoinThreads + tid, r = x / (D / 4);
            float total = 0.f;
#pragma unroll
            for (int p = 0; p < kSeats; ++p) total += sm.seat[p * kWideRows + r];
            finish_row<D, uint16_t>(a, row_of(a, s, group, h, r0 + r), (x - r * (D / 4)) * 4, sm.top[r], total, vscale, v[i]);
          }
        }
      }
    }
    tc_before();
    __syncthreads();                                          // the tile's memory is free again
    tc_after();
  }
  if (tid == 0 && sm.failed) set_err(a.err, PSPEC_DEVERR_WAIT);
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

template <int D>
cudaError_t launch_wide(AttendLaunch L, cudaStream_t stream) {
  constexpr int smem = sizeof(WideSmem<D>) + 1024;
  static_assert(2 * (smem + 1024) <= 227 * 1024, "two CTAs to an SM");
  auto* fn = attend_wide_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  L.ctas = kWideCtas;
  fn<<<L.ctas, kWideThreads, smem, stream>>>(L);
  return cudaGetLastError();
}

}  // namespace

size_t attend_wide_part_bytes() { return sizeof(float) * 2 * kWideCtas * Wide<128>::kPart; }

// Enough rows to a sequence that a tile of 128 costs less than several of 32 or 16, and tiles for
// half of the GPU (below that the narrow ones spread better).  32 sequences of 8192 keys, 8 kv
// heads, us by rows to a kv head (narrow, wide): D = 64, 32 rows 159, 158, 48 rows 234, 182, 128 rows
// 450, 193; D = 128, 32 rows 242, 302, 48 rows 346, 308, 128 rows 870, 332.
bool attend_is_wide(const AttendLaunch& L) {
  const long long rows = ((long long)L.a.T * (L.a.Hq / L.a.Hkv) + L.a.B - 1) / L.a.B;
  return L.a.dtype == PSPEC_BF16 && rows > (L.a.D == 64 ? 32 : 40) &&
         (long long)L.a.B * L.a.Hkv * ((rows + kWideRows - 1) / kWideRows) >= kNumSMs / 2;
}

cudaError_t launch_attend_wide(const AttendLaunch& L, cudaStream_t stream) {
  return L.a.D == 64 ? launch_wide<64>(L, stream) : launch_wide<128>(L, stream);
}

}  // namespace pspec
