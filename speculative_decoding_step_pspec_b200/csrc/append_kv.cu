// append_kv.cu -- keys and values into the paged cache, rotated to their positions (one
// launch), with the query rows rotated beside them.
//
// A CTA takes `rows_per_cta` rows.  Its threads first form the rows' angles pos * inv_freq in
// fp64 (positions reach 10^6: an fp32 product would be off by 0.06 rad there) and their sine
// and cosine, once for all heads; then every thread owns fixed elements of a head, keeps their
// coefficients in registers and walks the heads.
//
// 4-bit cache: four lanes share a block of 16 elements (four each); the block's largest
// magnitude goes round the four by shuffles.  Rotation and quantisation run in fp64: a value
// next to the border of two codes takes the wrong one when it is off by anything, and the
// borders mid * s * g (3 + 4 + 24 significant bits) are exact there, so no division is needed
// per element and ties are seen as ties.
#include "common.cuh"
#include "kernels.h"

namespace pspec {

namespace {

template <typename Tag> struct Row;
template <> struct Row<BF16Tag> {
  // 4 or 8 consecutive elements as floats; `vec`: the address is aligned to their size
  static __device__ __forceinline__ void load4(const uint16_t* p, bool vec, float (&x)[4]) {
    if (vec) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = __uint_as_float((uint32_t)p[j] << 16);
    }
  }
  static __device__ __forceinline__ uint16_t round(float x) {
    uint16_t r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
    return r;
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ void store4(uint16_t* p, bool vec, const float (&x)[4]) {
    if (vec) {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack(x[0], x[1]), pack(x[2], x[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = round(x[j]);
    }
  }
};
template <> struct Row<F32Tag> {
  static __device__ __forceinline__ void load4(const float* p, bool vec, float (&x)[4]) {
    if (vec) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = p[j];
    }
  }
  static __device__ __forceinline__ void store4(float* p, bool vec, const float (&x)[4]) {
    if (vec) {
      *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = x[j];
    }
  }
};

// The four consecutive elements j0 .. j0+3 that a thread owns in every head of one row: their
// coefficients, and where their partners are.
struct Turn {
  double c[4], s[4];   // out_j = x_j c + partner_j s (s carries the sign)
  int partner;         // offset of the partner of element 0; -1: inside the vector (x[j ^ 1])
  unsigned mask;       // bit j: element j0 + j is rotated
};

__device__ __forceinline__ Turn make_turn(const double2* cs, int j0, int rot, bool interleaved) {
  Turn t;
  const int h = rot >> 1;
  t.mask = 0;
  t.partner = -1;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int j = j0 + e;
    t.c[e] = 1.0;
    t.s[e] = 0.0;
    if (j < rot) {
      const double2 v = cs[interleaved ? j >> 1 : (j < h ? j : j - h)];
      const bool first = interleaved ? !(j & 1) : j < h;
      t.c[e] = v.x;
      t.s[e] = first ? -v.y : v.y;
      t.mask |= 1u << e;
    }
  }
  return t;
}

// The partners of elements j0 .. j0+3 of a head (half split): j + h below h, j - h from h on.
template <typename Tag>
__device__ __forceinline__ void load_partners(const typename Tag::elem* head, int j0, int rot,
                                              bool vec, float (&p)[4]) {
  const int h = rot >> 1;
  if ((h & 3) == 0) {
    Row<Tag>::load4(head + (j0 < h ? j0 + h : j0 - h), vec, p);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = j0 + e;
      p[e] = j < rot ? load_scalar(head, j < h ? j + h : j - h) : 0.f;
    }
  }
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

template <typename Tag, bool kE2M1>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendLaunch L) {
  using elem = typename Tag::elem;
  extern __shared__ double2 s_cs[];                   // [rows_per_cta][rot / 2] (cos, sin)
  const pspec_append_args& a = L.a;
  const int tid = threadIdx.x;
  const int h = a.rot >> 1;
  const long long t0 = (long long)blockIdx.x * L.rows_per_cta;
  const int rows = (int)min((long long)L.rows_per_cta, a.T - t0);

  for (int i = tid; i < rows * h; i += kThreads) {
    const int r = i / h, j = i - r * h;
    if (__ldg(a.slot_mapping + t0 + r) < 0) continue;
    double s, c;
    sincos((double)__ldg(a.positions + t0 + r) * (double)__ldg(a.inv_freq + j), &s, &c);
    s_cs[i] = make_double2(c, s);
  }
  __syncthreads();

  const int nl = a.D >> 2;                            // threads per head, four elements each
  const int groups = kThreads / nl;
  const int hg = tid / nl, j0 = (tid - hg * nl) * 4;
  const bool mine = hg < groups;
  const unsigned quad = 0xfu << (tid & 28);
  for (int r = 0; r < rows; ++r) {
    const long long t = t0 + r;
    const long long slot = __ldg(reinterpret_cast<const long long*>(a.slot_mapping) + t);
    if (slot < 0 || slot >= L.slots) {
      if (tid == 0 && slot != PSPEC_PADDING_SLOT_ID) set_err(a.err, PSPEC_DEVERR_BLOCK_RANGE);
      continue;
    }
    if (!mine) continue;
    const long long block = slot / a.block_size;
    const int off = (int)(slot - block * a.block_size);
    const Turn turn = make_turn(s_cs + r * h, j0, a.rot, a.interleaved != 0);

    // rotated in fp32: the result is rounded to the rows' dtype, no border to decide
    auto turned = [&](const elem* head, bool vec, float (&x)[4]) {
      Row<Tag>::load4(head + j0, vec, x);
      if (!turn.mask) return;
      float p[4];
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = x[e ^ 1];
      } else {
        load_partners<Tag>(head, j0, a.rot, vec, p);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (turn.mask >> e & 1) x[e] = fmaf(x[e], (float)turn.c[e], p[e] * (float)turn.s[e]);
    };

    if (a.q) {
      const elem* q = static_cast<const elem*>(a.q) + t * a.q_stride;
      elem* o = static_cast<elem*>(a.q_out) + t * (long long)a.Hq * a.D;
      for (int hd = hg; hd < a.Hq; hd += groups) {
        float x[4];
        turned(q + (long long)hd * a.D, L.vec_q, x);
        Row<Tag>::store4(o + (long long)hd * a.D + j0, L.vec_qo, x);
      }
    }

    const elem* kr = static_cast<const elem*>(a.k) + t * a.k_stride;
    const elem* vr = static_cast<const elem*>(a.v) + t * a.v_stride;
    for (int i = hg; i < 2 * a.Hkv; i += groups) {    // the key heads, then the value heads
      const bool is_k = i < a.Hkv;
      const int hd = is_k ? i : i - a.Hkv;
      const elem* head = (is_k ? kr : vr) + (long long)hd * a.D;
      const bool vec = is_k ? L.vec_k : L.vec_v;
      const long long row = (block * a.Hkv + hd) * a.block_size + off;   // row of the cache
      elem* echo = static_cast<elem*>(is_k ? a.k_out : a.v_out);
      if (echo) echo += (t * a.Hkv + hd) * a.D + j0;
      const bool vec_e = is_k ? L.vec_ko : L.vec_vo;
      if constexpr (!kE2M1) {
        float x[4];
        if (is_k) turned(head, vec, x);
        else Row<Tag>::load4(head + j0, vec, x);
        elem* dst = static_cast<elem*>(is_k ? a.k_pages : a.v_pages) + row * a.D + j0;
        Row<Tag>::store4(dst, true, x);
        if (echo) Row<Tag>::store4(echo, vec_e, x);
      } else {
        float xf[4];
        Row<Tag>::load4(head + j0, vec, xf);
        double x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = xf[e];
        if (is_k && turn.mask) {
          float p[4];
          if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = xf[e ^ 1];
          } else {
            load_partners<Tag>(head, j0, a.rot, vec, p);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (turn.mask >> e & 1) x[e] = fma((double)xf[e], turn.c[e], (double)p[e] * turn.s[e]);
        }
        double top = 0.0;
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmax(top, fabs(x[e]));   // drops NaN
        top = fmax(top, __shfl_xor_sync(quad, top, 1));
        top = fmax(top, __shfl_xor_sync(quad, top, 2));
        const float* scales = is_k ? a.k_scale : a.v_scale;
        const float g = scales ? __ldg(scales + hd) : 1.f;
        unsigned sc;
        const double s = e4m3_round(top / (double)g / 6.0, sc);
        const double u = s * (double)g;
        unsigned code[4], packed = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          code[e] = s > 0.0 ? e2m1_code(fabs(x[e]), u) : 0u;
          code[e] |= x[e] == x[e] && signbit(x[e]) ? 8u : 0u;
          packed |= code[e] << (4 * e);
        }
        uint8_t* pages = static_cast<uint8_t*>(is_k ? a.k_pages : a.v_pages);
        *reinterpret_cast<uint16_t*>(pages + row * (a.D >> 1) + (j0 >> 1)) = (uint16_t)packed;
        if ((j0 & 15) == 0) {
          uint8_t* bs = static_cast<uint8_t*>(is_k ? a.k_block_scales : a.v_block_scales);
          bs[row * (a.D >> 4) + (j0 >> 4)] = (uint8_t)sc;
        }
        if (echo) {                                   // level * s is exact, one rounding with g
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = e2m1_value(code[e]) * (float)s * g;
          Row<Tag>::store4(echo, vec_e, v);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_append(const AppendLaunch& L, cudaStream_t stream) {
  const unsigned grid = (unsigned)((L.a.T + L.rows_per_cta - 1) / L.rows_per_cta);
  const size_t smem = (size_t)L.rows_per_cta * (L.a.rot / 2) * sizeof(double2);
  const bool e2m1 = L.a.cache == PSPEC_CACHE_E2M1;
  if (L.a.dtype == PSPEC_BF16) {
    if (e2m1) append_kernel<BF16Tag, true><<<grid, kThreads, smem, stream>>>(L);
    else append_kernel<BF16Tag, false><<<grid, kThreads, smem, stream>>>(L);
  } else {
    if (e2m1) append_kernel<F32Tag, true><<<grid, kThreads, smem, stream>>>(L);
    else append_kernel<F32Tag, false><<<grid, kThreads, smem, stream>>>(L);
  }
  return cudaGetLastError();
}

}  // namespace pspec
