// Residual addition, root-mean-square norm and quantisation into the expert
// FFN's activation format, in one pass over the rows:
//
//   z = x + residual                     (fp32, not rounded before the norm)
//   residual_out = round(z)              (bf16, or fp32 as it is)
//   n = z * 1/sqrt(mean(z^2) + eps) * weight
//   x_norm = bf16(n)
//   x_q, x_sf = n quantised per block of 128 (E4M3, fp32 scale amax/448), 32
//               (E4M3, the smallest power of two 2^e with 448 * 2^e >= amax) or
//               16 columns (E2M1, E4M3 scale of amax / (6 x_gs))
//
// The formats are those of the MoEActivationPack page's encodings list and the
// quantisation rules those of the FFN's own intermediate.  A block that holds a
// NaN gets a NaN scale (the codes of such a block mean nothing), so that a NaN
// is never turned into a number on the way into the experts.
//
// The sum of squares and the root are fp64 and the products keep what they drop, so that n is rounded once, for any
// finite z that is not below 2^-100 of its row's rms.
//
// A workgroup owns one row, which stays in registers between the sum of squares
// and the outputs: thread i holds the 8-column chunks i, i + threads, ....  Each
// quantisation block then lies in 16, 4 or 2 neighbouring lanes, and its maximum
// takes DPP moves only.
//
// FP8 and NVFP4 codes are those of the quotient of n and the scale, each an fp32 number, rounded to fp32 and then to
// the code; MX codes those of n before any rounding.
//
// Bound by the bytes: 8192 x 7168 with residual, bf16 norm and FP8 codes moves 530 MB in 93 us (5.7 TB/s; a plain
// copy of 2 GiB reaches 4.9), NVFP4 codes 504 MB in 94 (5.4), 2048 x 2880 with an fp32 stream 89 MB in 16.2; one row
// by its latency, 3.4 us.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "layer.h"
#include "topk.h"

namespace moe {

namespace {

constexpr float kMinNormal = 1.17549435e-38f;

struct NormParams {
  const void* x;
  const void* residual;
  const void* weight;
  void* residual_out;
  void* x_norm;
  void* x_q;
  void* x_sf;
  int H;
  int weight_f32;
  float eps, x_gs;  // x_gs: NVFP4's global scale, times 2^x_exp
  int x_exp;
  double inv_h;
};

MOE_DEV void unpack8(i32x4 v, float (&f)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = __uint_as_float((uint32_t)v[q] << 16);
    f[2 * q + 1] = __uint_as_float((uint32_t)v[q] & 0xFFFF0000u);
  }
}
template <bool F32>
MOE_DEV void load8(const void* base, size_t i, float (&f)[8]) {
  if constexpr (F32) {
    const f32x4 a = *(const f32x4*)((const float*)base + i), b = *(const f32x4*)((const float*)base + i + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) f[q] = a[q], f[4 + q] = b[q];
  } else {
    unpack8(*(const i32x4*)((const uint16_t*)base + i), f);
  }
}
MOE_DEV i32x4 pack8(const float (&f)[8]) {
  i32x4 o;
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = (int)bf16x2_rne(f[2 * q], f[2 * q + 1]);
  return o;
}

// The rows' stores are non-temporal: the lines of the inputs, which other rows' loads share, stay
// (8192 x 7168: 97 -> 93 us, 512 x 7168: 9.1 -> 7.4; non-temporal loads were 8 to 30 % slower).
MOE_DEV void store16(void* p, i32x4 v) { __builtin_nontemporal_store(v, (i32x4*)p); }

// The largest |f| of 8 values, as bits: unsigned order puts NaN above infinity, so a NaN survives.
MOE_DEV uint32_t amax_bits8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}
// 1 / sqrt(m) in fp64: the row's codes share this factor, and each one that lies nearer to a rounding border
// than its error comes out as the other code.  Two Newton steps from the float root, or the fp64 root where m is
// no normal float.
MOE_DEV double inv_root(double m) {
  const float f = (float)m;
  if (!(f < INFINITY && f >= kMinNormal)) return 1.0 / sqrt(m);
  double r = (double)__builtin_amdgcn_rsqf(f);
  r = fma(0.5 * r, fma(-m * r, r, 1.0), r);
  return fma(0.5 * r, fma(-m * r, r, 1.0), r);
}
// v to odd: cut to 24 bits with the last one set if anything was cut.  Rounding that to fewer bits gives what
// rounding v itself would.
MOE_DEV float to_odd(double v) {
  const float f = (float)v;
  const double e = v - (double)f;
  const uint32_t u = __float_as_uint(f), cut = __builtin_islessgreater(e, 0.0) ? 1u : 0u;  // (an infinity's e is NaN)
  return __uint_as_float((u - ((u ^ (uint32_t)(__builtin_bit_cast(uint64_t, e) >> 32)) >> 31 & cut)) | cut);
}

// What one row's chunk writes of the format's activations: n the 8 values, c the chunk.
template <Fmt F>
MOE_DEV void quantise8(const NormParams& p, size_t t, int c, const float (&n)[8], bool live) {
  const int lane = lane_id(), C = p.H >> 3;
  if constexpr (F == Fmt::NVF4) {
    // an x_gs far from 1: n and x_gs both over its power of two, so that the scales' products and quotients are
    // normal numbers
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = n[i];
    if (p.x_exp != 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = __builtin_ldexpf(n[i], p.x_exp);
    }
    const float a = __uint_as_float(dpp_max_u32<0xB1>(amax_bits8(u)));  // lanes l, l ^ 1
    // v_cvt_pk_fp8_f32 past the E4M3 maximum would give NaN: the scale saturates; a NaN maximum stays one
    const float s6 = a / (6.0f * p.x_gs);
    const uint32_t code = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(s6 > 448.0f ? 448.0f : s6, 0.0f, 0, false) & 0xFFu;
    const float den = __builtin_amdgcn_cvt_f32_fp8((int)code, 0) * p.x_gs;
    const float inv = den > 0.0f ? 1.0f / den : 0.0f;
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the quotient u / den, rounded once, so that ties go to the even code (bounded, so that an infinite u keeps
      // its sign)
      float q = __builtin_amdgcn_fmed3f(u[i] * inv, 16.0f, -16.0f);
      q = fmaf(fmaf(-q, den, u[i]), inv, q);
      // magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6 -> codes 0 .. 7, in steps of 0.5, 1 and 2; ties to even
      const float b = fminf(fabsf(q), 6.0f);
      const float k = __builtin_rintf(b * (b < 2.0f ? 2.0f : b < 4.0f ? 1.0f : 0.5f)) + (b < 2.0f ? 0.0f : b < 4.0f ? 2.0f : 4.0f);
      v |= ((uint32_t)k | (k != 0.0f && q < 0.0f ? 8u : 0u)) << (4 * i);
    }
    if (live) {
      ((uint32_t*)p.x_q)[t * C + c] = v;
      if ((lane & 1) == 0) ((uint8_t*)p.x_sf)[t * (C >> 1) + (c >> 1)] = (uint8_t)code;
    }
    return;
  }
  uint32_t m = amax_bits8(n);
  m = dpp_max_u32<0xB1>(m);  // lanes l, l ^ 1
  m = dpp_max_u32<0x4E>(m);  // 4 lanes: 32 columns
  float inv, sc = 1.0f;
  if constexpr (F == Fmt::FP8) {
    m = dpp_max_u32<0x141>(m);
    m = dpp_max_u32<0x140>(m);  // 16 lanes: 128 columns
    const float a = __uint_as_float(m);
    // an all-zero block has scale 1; a scale below the smallest normal number would have no finite reciprocal
    const float s = a / 448.0f;
    sc = m == 0 ? 1.0f : (s < kMinNormal ? kMinNormal : s);
    inv = 1.0f / sc;
    if (live && (lane & 15) == 0) ((float*)p.x_sf)[t * (C >> 4) + (c >> 4)] = sc;
  } else {
    const bool nan = m > 0x7F800000u;
    const int e = mx_exponent_for_amax(__uint_as_float(m));
    inv = exp2i(-e);
    if (live && (lane & 3) == 0) ((uint8_t*)p.x_sf)[t * (C >> 2) + (c >> 2)] = nan ? (uint8_t)255 : (uint8_t)(e + 127);
  }
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = n[i] * inv;  // MX: exact
    // the quotient n / sc, rounded once (0 over an infinite scale)
    if constexpr (F == Fmt::FP8) q[i] = fmaf(fmaf(-q[i], fminf(sc, FLT_MAX), n[i]), inv, q[i]);
  }
  uint2 v;
  v.x = f32x2_to_e4m3_sat(q[0], q[1]) | f32x2_to_e4m3_sat(q[2], q[3]) << 16;
  v.y = f32x2_to_e4m3_sat(q[4], q[5]) | f32x2_to_e4m3_sat(q[6], q[7]) << 16;
  if (live) __builtin_nontemporal_store((uint64_t)v.y << 32 | v.x, (uint64_t*)p.x_q + t * C + c);
}

// NV: chunks a thread holds.  RES: 0 no residual, 1 bf16, 2 fp32.
template <Fmt F, int NV, bool XF32, int RES>
__global__ __launch_bounds__(1024) void add_rmsnorm_kernel(NormParams p) {
  __shared__ double part[16];
  const size_t t = blockIdx.x;
  const int tid = threadIdx.x, C = p.H >> 3, nthr = blockDim.x;
  float z[NV][8];
  double ss = 0.0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = tid + v * nthr;
    const size_t at = t * p.H + (size_t)c * 8;
    if (c < C) {
      load8<XF32>(p.x, at, z[v]);
      if constexpr (RES != 0) {
        float r[8];
        load8<RES == 2>(p.residual, at, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[v][i] += r[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[v][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma((double)z[v][i], (double)z[v][i], ss);
  }
  // (the row stays as floats: kept alive past the sum, its fp64 copies double the registers, 92 -> 105 us)
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("" : "+v"(z[v][i]));
  ss = wave_sum_f64(ss);
  double sum = ss;
  if (nthr > 64) {
    if ((tid & 63) == 0) part[tid >> 6] = ss;
    __syncthreads();
    sum = 0.0;
    for (int w = 0; w < nthr >> 6; ++w) sum += part[w];
  }
  const double r = inv_root(sum * p.inv_h + (double)p.eps);
  const float r_hi = (float)r, r_lo = (float)(r - (double)r_hi);
  // a row whose 1 / rms has no two full halves in fp32, or is 0, infinite or NaN
  const bool far = !(r_hi >= 0x1p-100f && r_hi <= 0x1p100f);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = tid + v * nthr;
    const bool live = c < C;
    const size_t at = t * p.H + (size_t)c * 8;
    float w[8] = {};
    if (live) {
      if (p.weight_f32) load8<true>(p.weight, (size_t)c * 8, w);
      else load8<false>(p.weight, (size_t)c * 8, w);
      if constexpr (RES == 1) store16((uint16_t*)p.residual_out + at, pack8(z[v]));
      if constexpr (RES == 2) {
        store16((float*)p.residual_out + at, __builtin_bit_cast(i32x4, f32x4{z[v][0], z[v][1], z[v][2], z[v][3]}));
        store16((float*)p.residual_out + at + 4, __builtin_bit_cast(i32x4, f32x4{z[v][4], z[v][5], z[v][6], z[v][7]}));
      }
    }
    // n = z r w, rounded once: what the products drop (r's lower half too) goes into the last one, an infinite w
    // does not
    float n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = z[v][i] * r_hi, lost = fmaf(z[v][i], r_lo, fmaf(z[v][i], r_hi, -a));
      n[i] = fmaf(a, w[i], lost * __builtin_amdgcn_fmed3f(w[i], FLT_MAX, -FLT_MAX));
    }
    bool again = far;
    if constexpr (F == Fmt::MX) {
      // MX codes are n times a power of two.  Where n's 24 bits end in a border of E4M3's codes (bit 19 alone of the
      // last 20: a tie of the normal ones; none of them: a tie of the subnormal ones, or 448, where the scale
      // changes; one in 2^19, a wave in 1000), what was rounded off decides.  (A subnormal n is left as it is.)
      uint32_t low = ~0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) low = min(low, __float_as_uint(n[i]) << 13);
      if (low == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) again |= (__float_as_uint(n[i]) << 13) == 0 && n[i] != 0.0f;
      }
    }
    if (again) {  // (fp64 for every row: 8192 x 7168 92.2 -> 94.7 us)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double d = (double)z[v][i] * r * (double)w[i];
        n[i] = F == Fmt::MX ? to_odd(d) : (float)d;
      }
    }
    if (live && p.x_norm != nullptr) store16((uint16_t*)p.x_norm + at, pack8(n));
    if constexpr (F != Fmt::BF16) quantise8<F>(p, t, c, n, live);
  }
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  NormParams p{a.x, a.residual, a.weight, a.residual_out, a.x_norm, a.x_q, a.x_sf, a.H, a.weight_f32 ? 1 : 0,
               a.eps, a.x_gs, 0, 1.0 / a.H};
  if (a.fmt == Fmt::NVF4 && !(a.x_gs > 0x1p-100f && a.x_gs < 0x1p100f)) {  // (finite and > 0)
    p.x_exp = -std::ilogb(a.x_gs);
    p.x_gs = std::ldexp(a.x_gs, p.x_exp);
  }
  const int chunks = a.H / 8;
  // Chunks per thread: one where the row fits 1024 threads (one row, H 7168, in a graph: 3.75 us, with two 4.3, with
  // four 5.4), two for wide rows by the thousand (8192 x 7168: 92.7 us, with one 95.2, with four 99.7).
  const int nv = chunks <= 512 || (chunks <= 1024 && a.T < 1024) ? 1 : chunks <= 2048 ? 2 : 4;
  const int threads = ((chunks + nv - 1) / nv + 63) / 64 * 64;
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3((unsigned)a.T), dim3((unsigned)threads), 0, s, p); };
  auto by_nv = [&](auto f, auto xf, auto res) {
    constexpr Fmt F = decltype(f)::value;
    constexpr bool X = decltype(xf)::value;
    constexpr int R = decltype(res)::value;
    if (nv == 1) go(add_rmsnorm_kernel<F, 1, X, R>);
    else if (nv == 2) go(add_rmsnorm_kernel<F, 2, X, R>);
    else go(add_rmsnorm_kernel<F, 4, X, R>);
  };
  auto by_type = [&](auto f) {
    auto by_res = [&](auto xf) {
      if (a.residual == nullptr) by_nv(f, xf, std::integral_constant<int, 0>{});
      else if (!a.residual_f32) by_nv(f, xf, std::integral_constant<int, 1>{});
      else by_nv(f, xf, std::integral_constant<int, 2>{});
    };
    if (a.x_f32) by_res(std::true_type{});
    else by_res(std::false_type{});
  };
  if (a.x_q == nullptr) by_type(std::integral_constant<Fmt, Fmt::BF16>{});
  else if (a.fmt == Fmt::FP8) by_type(std::integral_constant<Fmt, Fmt::FP8>{});
  else if (a.fmt == Fmt::MX) by_type(std::integral_constant<Fmt, Fmt::MX>{});
  else by_type(std::integral_constant<Fmt, Fmt::NVF4>{});
  return hipGetLastError();
}

}  // namespace moe
