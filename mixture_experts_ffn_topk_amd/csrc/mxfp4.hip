// MXFP4 quantisation of rows, and the clamped SwiGLU between the experts' two products: forward to bf16 and to MXFP4, and
// backward.
//
//   MXFP4     per 32 columns the smallest e in [-127, 127] with 6 * 2^e >= amax; codes E2M1_RNE_sat(x / 2^e), the scale
//             byte e + 127.  x / 2^e is a change of exponent, so the codes are the roundings of x itself.
//   SwiGLU    g' = min(g, c), u' = clamp(u, -c, c), s = 1 / (1 + e^-g'):  h = g' s u'
//   backward  dg = dh u' s (1 + g' (1 - s)) where g <= c, du = dh g' s where |u| <= c, else 0
//
// A thread holds 8 columns (16 bytes of bf16), four neighbouring lanes a block of 32.  Everything is read once and written
// once, so memory bounds all of it.
#include <algorithm>

#include "gemm_common.h"
#include "grouped.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------- MXFP4
// The exponent for a block whose largest magnitude has these bits (6 = 1.5 * 2^2: one more where the significand passes
// 1.5).  Subnormals take -127: 6 * 2^-127 is above them all; an infinity takes the largest, 127.
MOE_DEV int mxfp4_exponent(uint32_t bits) {
  const int e = (int)(bits >> 23) - 129 + ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return (bits >> 23) == 0 ? -127 : (bits >> 23) == 255 ? 127 : max(e, -127);
}

struct Mxfp4 {
  uint32_t codes;  // 8 of them
  int scale;       // the block's byte: e + 127, or 255 for a block that holds a NaN
};
// Eight columns of a block that lanes 4 i .. 4 i + 3 hold.
MOE_DEV Mxfp4 mxfp4_of(const float (&v)[8]) {
  // magnitudes compare as integers, and a NaN's is above infinity's
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  top = max(top, (uint32_t)__shfl_xor((int)top, 1));
  top = max(top, (uint32_t)__shfl_xor((int)top, 2));
  const int e = mxfp4_exponent(top);
  // (the conversion divides by its scale's power of two, rounds to nearest even and saturates; small blocks are raised
  // first, so that neither the values nor the scale are subnormal)
  const bool small = e < -60;
  const float raise = small ? 0x1p64f : 1.0f, scale = __uint_as_float((uint32_t)(e + 127 + (small ? 64 : 0)) << 23);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * raise, v[1] * raise, scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * raise, v[3] * raise, scale, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * raise, v[5] * raise, scale, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * raise, v[7] * raise, scale, 3);
  return Mxfp4{c, top > 0x7F800000u ? 255 : e + 127};
}
MOE_DEV void mxfp4_store(const Mxfp4& m, void* q, void* sf, long long chunk) {
  ((uint32_t*)q)[chunk] = m.codes;
  if ((chunk & 3) == 0) ((uint8_t*)sf)[chunk >> 2] = (uint8_t)m.scale;
}
// What the codes stand for, in bf16 (exact but for 2^128 and above, 4 * 2^126 say, which are infinities).
MOE_DEV i32x4 mxfp4_values(const Mxfp4& m) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const float s = m.scale == 255 ? __uint_as_float(0x7FC00000u) : exp2i(m.scale - 127);
  const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(m.codes, 1.0f, 0),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(m.codes, 1.0f, 1),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(m.codes, 1.0f, 2),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(m.codes, 1.0f, 3)};
  i32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (int)bf16x2_rne(p[i][0] * s, p[i][1] * s);
  return r;
}

MOE_DEV void unpack8(const i32x4 a, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float((uint32_t)a[i] << 16);
    v[2 * i + 1] = __uint_as_float((uint32_t)a[i] & 0xFFFF0000u);
  }
}
MOE_DEV i32x4 pack8(const float (&v)[8]) {
  i32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (int)bf16x2_rne(v[2 * i], v[2 * i + 1]);
  return r;
}

struct QuantParams {
  const void* x;
  long long rows;  // 1 where the rows lie one behind the other
  long long chunks, stride;  // chunks of 8 a row; elements between rows
  void* q;
  void* sf;
  void* values;
};

template <bool F32>
__global__ __launch_bounds__(kThreads) void quantize_mxfp4_kernel(QuantParams p) {
  for (long long row = blockIdx.y; row < p.rows; row += gridDim.y) {
    for (long long c = (long long)blockIdx.x * kThreads + threadIdx.x; c < p.chunks; c += (long long)gridDim.x * kThreads) {
      float v[8];
      if constexpr (F32) {
        const f32x4* x = (const f32x4*)((const float*)p.x + row * p.stride + c * 8);
        const f32x4 a = x[0], b = x[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
      } else {
        unpack8(*(const i32x4*)((const uint16_t*)p.x + row * p.stride + c * 8), v);
      }
      const Mxfp4 m = mxfp4_of(v);
      mxfp4_store(m, p.q, p.sf, row * p.chunks + c);
      if (p.values) ((i32x4*)p.values)[row * p.chunks + c] = mxfp4_values(m);
    }
  }
}

// ---------------------------------------------------------------- SwiGLU
// Finite where an infinite gate meets a zero: below its sigmoid's, above that of the backward pass's g' (1 - s) alone (the
// value there is the infinity).  A NaN stays one.
constexpr float kTop = 3.402823466e38f;
MOE_DEV float finite_below(float g) { return g < -kTop ? -kTop : g; }
MOE_DEV float finite_above(float g) { return g > kTop ? kTop : g; }
// t = e^(-|g| / 2): its square may be subnormal where what it is multiplied by is not, so neither the square nor g' times it is
// formed alone.  (t itself is normal down to g = -174.  Below, only up columns past 2^112 would give more than bf16's zero.)
template <bool FAST>
MOE_DEV float half_exp(float g) {
  return FAST ? __builtin_amdgcn_exp2f(fabsf(g) * -0.7213475204444817f) : expf(fabsf(g) * -0.5f);
}
template <bool FAST>
MOE_DEV float inverse(float v) {
  return FAST ? __builtin_amdgcn_rcpf(v) : 1.0f / v;
}

template <bool BACK, bool FAST>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(SwigluArgs p) {
  const int per_row = p.I / 8, valid = min(max(p.start[p.E], 0), p.npairs);
  // rows narrower than the workgroup share it
  const int together = max(1, kThreads / per_row), mine = threadIdx.x / per_row;
  const long long row = (long long)blockIdx.x * together + (together > 1 ? mine : 0);
  if (row >= valid || (together > 1 && mine >= together)) return;
  const int c0 = together > 1 ? threadIdx.x - mine * per_row : threadIdx.x, step = together > 1 ? per_row : kThreads;
  const i32x4* gu = (const i32x4*)((const uint16_t*)p.gu + row * 2 * p.I);
  for (int c = c0; c < per_row; c += step) {
    float g[8], u[8], d[8], o[8];
    unpack8(gu[c], g);
    unpack8(gu[per_row + c], u);
    if constexpr (BACK) unpack8(((const i32x4*)((const uint16_t*)p.dh + row * p.I))[c], d);
    float dg[8], du[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // (comparisons, not fminf: a NaN stays one)
      const float gc = finite_below(g[i] > p.clamp ? p.clamp : g[i]);
      const float uc = u[i] > p.clamp ? p.clamp : u[i] < -p.clamp ? -p.clamp : u[i];
      // s = t^2 / (1 + t^2) below zero, 1 / (1 + t^2) above
      const float t = half_exp<FAST>(gc), r = inverse<FAST>(fmaf(t, t, 1.0f)), f = gc < 0.0f ? t : 1.0f;
      const float fr = f * r, a = gc * fr;
      o[i] = a * (f * uc);
      if constexpr (BACK) {
        const float s = fr * f;
        dg[i] = g[i] > p.clamp ? 0.0f : d[i] * uc * fr * fmaf(finite_above(gc), 1.0f - s, 1.0f) * f;
        du[i] = fabsf(u[i]) > p.clamp ? 0.0f : a * (f * d[i]);
      }
    }
    const long long chunk = row * per_row + c;
    if constexpr (BACK) {
      i32x4* out = (i32x4*)((uint16_t*)p.dgu + row * 2 * p.I);
      out[c] = pack8(dg);
      out[per_row + c] = pack8(du);
    } else if (p.q) {
      mxfp4_store(mxfp4_of(o), p.q, p.sf, chunk);
    }
    if (p.h) ((i32x4*)p.h)[chunk] = pack8(o);
  }
}

}  // namespace

hipError_t launch_quantize_mxfp4(const void* x, bool x_f32, long long rows, int cols, long long stride, void* q, void* sf,
                                 void* values, hipStream_t s) {
  if (rows <= 0) return hipSuccess;
  QuantParams p{x, rows, cols / 8, stride, q, sf, values};
  if (stride == cols) p.chunks *= rows, p.rows = 1;
  const long long blocks = (p.chunks + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)std::min(blocks, 1LL << 20), (unsigned)std::min(p.rows, 32768LL));
  if (x_f32)
    quantize_mxfp4_kernel<true><<<grid, dim3(kThreads), 0, s>>>(p);
  else
    quantize_mxfp4_kernel<false><<<grid, dim3(kThreads), 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s) {
  const int together = std::max(1, kThreads / (a.I / 8));
  const long long blocks = ((long long)a.npairs + together - 1) / together;
  if (blocks <= 0) return hipSuccess;
  const dim3 grid((unsigned)blocks), block(kThreads);
  if (a.dgu) {
    if (a.fast)
      swiglu_kernel<true, true><<<grid, block, 0, s>>>(a);
    else
      swiglu_kernel<true, false><<<grid, block, 0, s>>>(a);
  } else if (a.fast) {
    swiglu_kernel<false, true><<<grid, block, 0, s>>>(a);
  } else {
    swiglu_kernel<false, false><<<grid, block, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace moe
