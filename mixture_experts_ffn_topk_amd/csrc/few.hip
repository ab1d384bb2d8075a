// The routed layer for few tokens (at most kFewMaxTokens) in two launches:
//
//   few_gate_up: routing (from logits, or the caller's ids) -> gate/up product of
//                every active expert -> clamped SwiGLU -> h
//   few_down:    requantised h -> down product -> router-weighted combine with the
//                addends -> out
//
// The same operator as moe_forward on the same prepared weights, for batches so
// small that the step is one pass over the active experts' weights.  What differs
// from the grouped GEMMs:
//   * The weights are the first MFMA operand (16 rows), an expert's tokens (in token
//     order, found from one 32-bit mask per expert in LDS) the 16 columns of the
//     second: no plan, no gathered rows.  An expert with more than 16 tokens is two
//     units of work that read its weights twice.  gate_up's workgroups each find
//     their unit from the ids; one more workgroup writes all units' tables for the
//     down launch, whose start is then one load away.
//   * Weights go straight from HBM into registers, each byte read once per unit, non-temporal,
//     and nothing is staged in LDS: a wave is on its own until its sums are complete.
//   * gate_up: a wave owns 16 or 32 columns of h (MX: 32, one scale block) of one expert,
//     or (all but FP8's whole blocks) 1/KSP of their K-steps.
//   * down: a workgroup owns 16 R output columns and all units, or one of `splits`
//     parts of them; its waves split its (unit, K-step) sequence evenly and add each
//     unit's result to their own sums per token in LDS: no y rows, no combine launch.
//     The splits' sums meet in the workspace: the last to arrive at a counter (which
//     gate_up zeroed) adds them in order.
//   * The FP8 intermediate needs the maximum over 128 columns.  Where whole 128-column
//     blocks make enough workgroups, the eight waves of a gate_up workgroup hold one
//     block and quantise it; otherwise (one token, small I) h stays fp32 between the
//     launches and every down workgroup quantises all of it into LDS first.  The
//     other formats' blocks lie inside one wave and are quantised there.
//
// Every expert's term is a fresh MFMA partial scaled by (router weight x block
// scales) in fp32, so the output is one fp32 sum per element, rounded once; the
// order of the sum is fixed by the sizes and the routing alone.
//
// The MFMAs of 8-bit operands add their 128 products to about 14 bits, as in moe_forward (block-scaled operands have
// no other form): a code of h at a midpoint may be its neighbour, which the outputs' tolerance counts.
//
// Bound by the weights' bytes, except NVFP4's decode (VALU).  Kernel times and rates: FP8, T 16, H 7168, I 2048,
// E 32, k 8: gate_up 920 MB in 146 us (6.3 TB/s), down 460 MB in 71.5 (6.4); T 1: 235 MB in 37 (6.4), 117 MB in 22.5
// (5.2), I 256 29 MB in 11.6, 15 MB in 6.5 (the start: routing, tables, masks, before the first weight); BF16, T 4,
// H 4096, I 14336: 1096 MB in 174 (6.3), 548 MB in 89 (6.2); W4A8, T 32, H 2880, E 128: 749 MB in 112 (6.7), 375 MB
// in 61.5 (6.1); NVFP4 x BF16, T 3: 242 MB in 46 (5.25), 121 MB in 27 (4.5); NVFP4 x NVFP4, T 32: 528 MB in 88 (6.0),
// 264 MB in 61 (4.4).  A read alone reaches 6.85 TB/s from 0.9 GB on, 6.4 at 0.24 GB.  An expert with more than 16
// tokens costs its weights twice: BF16, H 4096, I 14336, E 8, T 32, k 2 (none) 440 us, k 8 (all) 1008; moe_forward
// 489 and 514.
#include <algorithm>
#include <type_traits>

#include "gemm_common.h"
#include "layer.h"
#include "topk.h"

namespace moe {

namespace {

constexpr int kFewMaxPairs = kFewMaxTokens * 32;  // num_topk <= 32
constexpr int kFewMaxExperts = 1024;
// (an expert with more than 16 of T <= 32 tokens is two units: at most one such per 17 pairs)
constexpr int few_max_units(int E, int T, int topk) {
  return (E < T * topk ? E : T * topk) + (T > 16 ? T * topk / 17 : 0);
}
constexpr int kFewMaxSplits = 8;
// FP8: the most bytes of h (with 16 spare ones per row) that the down launch quantises into LDS: two
// workgroups still share a CU.
constexpr int kFewLdsH = 48 * 1024;

// 16-bit operands on the matrix cores, and a 16-bit h
constexpr bool mma16(Fmt f) { return f == Fmt::BF16 || f == Fmt::NV4 || f == Fmt::NVF4; }
constexpr bool nv4w(Fmt f) { return f == Fmt::NV4 || f == Fmt::NVF4; }

struct FewParams {
  int T, topk, E, H, I;
  int fast;
  float clamp;
  const void* ids;  // [T, k]
  int ids64;
  const float* topk_w;
  const float* logits;  // gate_up: route here (nullptr: ids are given)
  const float* bias;
  int* idx32_out;       // where the routing goes (one of them), and its weights
  long long* idx64_out;
  float* w_out;
  const uint8_t* x;
  const uint8_t* x_sf;
  uint32_t x_row, x_sf_row;  // bytes
  const uint8_t* w;     // the leg's prepared weights
  const uint8_t* w_sf;
  uint32_t w_expert, w_sf_expert;  // bytes per expert
  const float* w_gs;
  const float* c_gs;
  int ksteps;           // K-steps of the prepared layout
  int steps;            // K-steps of the kernel (NVFP4: pairs of the layout's)
  void* h;
  void* h_sf;
  uint32_t* tables;     // the units (FewTables)
  int max_units;
  int splits;           // down: workgroups that share a block of columns
  int n_blocks;         // down: blocks of 16 R columns
  int* arrived;         // [n_blocks]
  float* part;          // [splits][n_blocks][R][T][16]
  const uint16_t* shared;
  const uint16_t* residual;
  void* out;
  int out_f32;
};

// ---------------------------------------------------------------- operands
typedef float f32x2 __attribute__((ext_vector_type(2)));
MOE_DEV int pack2(f32x2 v) { return (int)bf16x2_rne(v[0], v[1]); }
// 8 E2M1 values (element 2i in the low nibble of byte i) times their E4M3 block
// scale, as bf16: the product of a 2-bit and a 4-bit significand is exact.
MOE_DEV i32x4 e2m1_bf16x8(uint32_t d, float s) {
  i32x4 r;
  r[0] = pack2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 0) * s);
  r[1] = pack2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 1) * s);
  r[2] = pack2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 2) * s);
  r[3] = pack2(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 3) * s);
  return r;
}
// The same as fp16, for NVFP4 x NVFP4: 6-bit products between 2^-10 and 6 x 448 are exact there too,
// and the packed product takes half the VALU operations (T 3, H 7168, I 2048, E 32, k 8: 103 us, this 90).
// Scale B of the four in sc (pairs).
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
template <int B>
MOE_DEV i32x4 e2m1_f16x8(uint32_t d, const f16x2 (&sc)[2]) {
  const f16x2 s = __builtin_shufflevector(sc[B >> 1], sc[B >> 1], B & 1, B & 1);
  i32x4 r;
  r[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 0) * s);
  r[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 1) * s);
  r[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 2) * s);
  r[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 3) * s);
  return r;
}
MOE_DEV void e4m3_f16x4(int v, f16x2 (&sc)[2]) {
  sc[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, false);
  sc[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.0f, true);
}
template <int B>
MOE_DEV float e4m3_byte(int v) {
  return __builtin_amdgcn_cvt_f32_fp8(v, B);
}
MOE_DEV i32x8 join(i32x4 a, i32x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }
MOE_DEV f32x4 mma_bf16(i32x4 w, i32x4 x, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
}

MOE_DEV f32x4 mma_f16(i32x4 w, i32x4 x, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x), c, 0, 0, 0);
}

// One K-step of a 16-row weight tile in registers.
//   FP8: q[0], q[1] the two 16-byte pieces; BF16: likewise, the two 32-element halves;
//   MX: q[0], s the scale byte; NVFP4: q[0] two of the layout's K-steps (lanes g = 0, 1
//   the first, 2, 3 the second), s the four E4M3 block scales of the lane's row.
template <Fmt F>
struct WFrag {
  i32x4 q[F == Fmt::FP8 || F == Fmt::BF16 ? 2 : 1];
  int s;
};
// The lane's part of a weight tile's address: row block rb (16 rows; the 32-row
// tiles of the bf16 formats: tile rb / 2, half rb % 2), relative to the expert.
template <Fmt F>
struct WAddr {
  uint32_t q, s;
};
template <Fmt F>
MOE_DEV WAddr<F> w_addr(int tile32, int half, int rb, int ksteps, int g, int r16, bool ok) {
  WAddr<F> a{};
  if constexpr (F == Fmt::FP8) {
    a.q = (uint32_t)rb * (uint32_t)ksteps * 2048u + 16u * (16 * g + r16);
  } else if constexpr (F == Fmt::MX) {
    a.q = (uint32_t)rb * (uint32_t)ksteps * 1024u + 16u * (16 * g + r16);
    a.s = (uint32_t)rb * (uint32_t)ksteps * 64u + (uint32_t)(16 * g + r16);
  } else if constexpr (F == Fmt::BF16) {
    // lane (g, r) of the 16x16x32 operand: sub-step 2q + g / 2, half-step g % 2 of tile row r
    a.q = (uint32_t)tile32 * (uint32_t)ksteps * 4096u + 1024u * (g >> 1) + 16u * (32 * (g & 1) + 16 * half + r16);
  } else {
    a.q = ((uint32_t)tile32 * (uint32_t)ksteps + (g >> 1)) * 1024u + 16u * (32 * (g & 1) + 16 * half + r16);
    a.s = ((uint32_t)tile32 * (uint32_t)ksteps + (g >> 1)) * 128u + 4u * (16 * half + r16);
  }
  if (!ok) a.q = a.s = kOOB;
  return a;
}
template <Fmt F>
MOE_DEV void w_load(WFrag<F>& f, const WAddr<F>& a, __amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t srs, int k,
                    uint32_t dead, int ksteps, int g) {
  if constexpr (F == Fmt::FP8) {
    f.q[0] = bload16_nt(rs, a.q | dead, (uint32_t)k * 2048u);
    f.q[1] = bload16_nt(rs, (a.q + 1024u) | dead, (uint32_t)k * 2048u);
  } else if constexpr (F == Fmt::MX) {
    f.q[0] = bload16_nt(rs, a.q | dead, (uint32_t)k * 1024u);
    f.s = (int)__builtin_amdgcn_raw_buffer_load_b8(srs, a.s | dead, (uint32_t)k * 64u, 0);
  } else if constexpr (F == Fmt::BF16) {
    f.q[0] = bload16_nt(rs, a.q | dead, (uint32_t)k * 4096u);
    f.q[1] = bload16_nt(rs, (a.q + 2048u) | dead, (uint32_t)k * 4096u);
  } else {
    dead |= oob_if(2 * k + (g >> 1) >= ksteps);  // an odd count of the layout's K-steps
    f.q[0] = bload16_nt(rs, a.q | dead, (uint32_t)k * 2048u);
    f.s = (int)__builtin_amdgcn_raw_buffer_load_b32(srs, a.s | dead, (uint32_t)k * 256u, 0);
  }
}

// One K-step of a 16-token activation slice.  v: FP8 / MX E4M3 bytes [16g, 16g+16) and
// [64+16g, ..) of the step's 128; BF16 the two 32-element halves; NVFP4 x BF16 the four
// sub-steps' 8 elements; NVFP4 x NVFP4 their packed codes in v[0].  s: the FP8 scale's
// bits, the MX scale byte, or NVFP4's four block scales.
template <Fmt F, bool GATEUP>
struct XFrag {
  static constexpr bool kPacked = F == Fmt::NVF4 && GATEUP;
  i32x4 v[nv4w(F) && !kPacked ? 4 : (kPacked ? 1 : 2)];
  int s;
};

// acc += (weights x activations) of one K-step; FP8: a partial, its scales are the caller's.
template <Fmt F, bool GATEUP>
MOE_DEV f32x4 mma_step(const WFrag<F>& w, const XFrag<F, GATEUP>& x, f32x4 acc) {
  if constexpr (F == Fmt::FP8) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(w.q[0], w.q[1]), join(x.v[0], x.v[1]), acc, 0, 0, 0,
                                                            127, 0, 127);
  } else if constexpr (F == Fmt::MX) {
    const i32x8 b8 = {w.q[0][0], w.q[0][1], w.q[0][2], w.q[0][3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b8, join(x.v[0], x.v[1]), acc, 4, 0, 0, w.s, 0, x.s);
  } else if constexpr (F == Fmt::BF16) {
    acc = mma_bf16(w.q[0], x.v[0], acc);
    return mma_bf16(w.q[1], x.v[1], acc);
  } else if constexpr (F == Fmt::NVF4) {
    f16x2 ws[2], xc[2];
    e4m3_f16x4(w.s, ws);
    if constexpr (GATEUP) {
      e4m3_f16x4(x.s, xc);
      acc = mma_f16(e2m1_f16x8<0>((uint32_t)w.q[0][0], ws), e2m1_f16x8<0>((uint32_t)x.v[0][0], xc), acc);
      acc = mma_f16(e2m1_f16x8<1>((uint32_t)w.q[0][1], ws), e2m1_f16x8<1>((uint32_t)x.v[0][1], xc), acc);
      acc = mma_f16(e2m1_f16x8<2>((uint32_t)w.q[0][2], ws), e2m1_f16x8<2>((uint32_t)x.v[0][2], xc), acc);
      return mma_f16(e2m1_f16x8<3>((uint32_t)w.q[0][3], ws), e2m1_f16x8<3>((uint32_t)x.v[0][3], xc), acc);
    } else {
      acc = mma_f16(e2m1_f16x8<0>((uint32_t)w.q[0][0], ws), x.v[0], acc);
      acc = mma_f16(e2m1_f16x8<1>((uint32_t)w.q[0][1], ws), x.v[1], acc);
      acc = mma_f16(e2m1_f16x8<2>((uint32_t)w.q[0][2], ws), x.v[2], acc);
      return mma_f16(e2m1_f16x8<3>((uint32_t)w.q[0][3], ws), x.v[3], acc);
    }
  } else {
    acc = mma_bf16(e2m1_bf16x8((uint32_t)w.q[0][0], e4m3_byte<0>(w.s)), x.v[0], acc);
    acc = mma_bf16(e2m1_bf16x8((uint32_t)w.q[0][1], e4m3_byte<1>(w.s)), x.v[1], acc);
    acc = mma_bf16(e2m1_bf16x8((uint32_t)w.q[0][2], e4m3_byte<2>(w.s)), x.v[2], acc);
    return mma_bf16(e2m1_bf16x8((uint32_t)w.q[0][3], e4m3_byte<3>(w.s)), x.v[3], acc);
  }
}

// ---------------------------------------------------------------- routing in LDS
struct RouteLds {
  short ids[kFewMaxPairs];        // expert of each pair, -1: no valid expert
  uint32_t mask[kFewMaxExperts];  // the tokens of each expert
};
constexpr int kCol(int t, int j) { return t << 5 | j; }  // a column: token and slot (both below 32)

// The pairs' experts and the experts' tokens, by the whole workgroup (ends with a barrier).
// from_logits (gate_up): each wave routes tokens wave, wave + WAVES, ...; w (the tables' workgroup,
// else nullptr) receives the router weights, and the caller's arrays the result.
template <int WAVES>
MOE_DEV void route_to_lds(const FewParams& p, RouteLds& L, float* w) {
  const int tid = threadIdx.x, lane = lane_id(), np = p.T * p.topk;
  auto id_of = [&](int q) { return p.ids64 ? ((const long long*)p.ids)[q] : (long long)((const int*)p.ids)[q]; };
  const bool routes = p.logits != nullptr;
  long long first = -1;  // (in flight while the masks are cleared)
  if (!routes && tid < np) first = id_of(tid);
  for (int e = tid; e < p.E; e += 64 * WAVES) L.mask[e] = 0;
  __syncthreads();
  if (routes) {
    for (int t = tid >> 6; t < p.T; t += WAVES) {
      int e;
      float wt;
      const float* row = p.logits + (size_t)t * p.E;
      if (p.fast) route_token_topk<true>(row, p.bias, p.E, p.topk, e, wt);
      else route_token_topk<false>(row, p.bias, p.E, p.topk, e, wt);
      if (lane < p.topk) {
        const int q = t * p.topk + lane;
        L.ids[q] = (short)e;
        atomicOr(&L.mask[e], 1u << t);
        if (w != nullptr) {
          if (p.idx64_out != nullptr) p.idx64_out[q] = e;
          else p.idx32_out[q] = e;
          p.w_out[q] = wt;
          w[q] = wt;
        }
      }
    }
  } else {
    for (int q = tid; q < np; q += 64 * WAVES) {
      const long long v = q == tid ? first : id_of(q);
      const bool ok = v >= 0 && v < p.E;
      L.ids[q] = ok ? (short)v : (short)-1;
      if (ok) atomicOr(&L.mask[(int)v], 1u << (q / p.topk));
      if (w != nullptr) w[q] = p.topk_w[q];
    }
  }
  __syncthreads();
}
MOE_DEV int bits_below(uint64_t b) {  // set bits of the lanes below this one
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(b >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)b, 0));
}
// Units of work: an active expert, or each half of one with more than 16 tokens, in expert order.
// Calls f(units before the lane's expert, the lane's expert, its units) for 64 experts at a time
// until f returns true; returns the number of units seen.
template <typename Fn>
MOE_DEV int for_units(const RouteLds& L, int E, Fn f) {
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane_id(), n = e < E ? __popc(L.mask[e]) : 0;
    const uint64_t b1 = __ballot(n > 0), b2 = __ballot(n > 16);
    if (f(base + bits_below(b1) + bits_below(b2), e, (n > 0 ? 1 : 0) + (n > 16 ? 1 : 0))) break;
    base += __popcll(b1) + __popcll(b2);
  }
  return base;
}
MOE_DEV int rank_in(uint32_t mask, int t) { return __popc(mask & ((1u << t) - 1u)); }

// The tables of the units for the down launch: the pairs' router weights (of a token's first slot
// of an expert: the sum over its slots of that expert, in slot order), each unit's expert and number of
// columns, and their columns.
struct FewTables {
  uint32_t *n, *w, *unit, *col;  // [4] (one used), [pairs] floats, [max_units], [max_units][8] pairs of shorts
};
MOE_HOST_DEV inline size_t few_table_words(int pairs, int max_units) { return 4 + (size_t)pairs + 9 * (size_t)max_units; }
MOE_DEV FewTables few_tables(uint32_t* base, int pairs, int max_units) {
  return FewTables{base, base + 4, base + 4 + pairs, base + 4 + pairs + max_units};
}
template <int WAVES>
MOE_DEV void write_tables(const FewParams& p, const RouteLds& L, const float* w, short* ustart) {
  const int tid = threadIdx.x, np = p.T * p.topk;
  const FewTables tb = few_tables(p.tables, np, p.max_units);
  if (tid < 64) {
    const int n = for_units(L, p.E, [&](int before, int e, int units) {
      const int cnt = units > 0 ? __popc(L.mask[e]) : 0;
      if (units > 0) {
        ustart[e] = (short)before;
        tb.unit[before] = (uint32_t)(e | min(cnt, 16) << 16);
      }
      if (units > 1) tb.unit[before + 1] = (uint32_t)(e | (cnt - 16) << 16);
      return false;
    });
    if (tid == 0) *tb.n = (uint32_t)n;
  }
  __syncthreads();
  for (int q = tid; q < np; q += 64 * WAVES) {
    const int e = L.ids[q], t = q / p.topk, j = q - t * p.topk;
    if (e < 0) continue;
    float s = 0.0f;
    bool first = true;
    for (int i = 0; i < p.topk; ++i)
      if (L.ids[t * p.topk + i] == e) {
        first = first && i >= j;
        s += w[t * p.topk + i];
      }
    if (!first) continue;
    const int r = rank_in(L.mask[e], t);
    ((float*)tb.w)[q] = s;
    ((short*)tb.col)[(ustart[e] + (r >> 4)) * 16 + (r & 15)] = (short)kCol(t, j);
  }
}

// ---------------------------------------------------------------- gate_up
// min and max that keep a NaN
MOE_DEV float clamp_hi(float v, float c) { return v > c ? c : v; }
MOE_DEV float clamp_both(float v, float c) { return v > c ? c : (v < -c ? -c : v); }
MOE_DEV f32x4 swiglu4(f32x4 g, f32x4 u, float c, int fast) {
  f32x4 h;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float gc = clamp_hi(g[i], c), uc = clamp_both(u[i], c);
    h[i] = (fast ? silu_f32<true>(gc) : silu_f32<false>(gc)) * uc;
  }
  return h;
}
MOE_DEV uint32_t amax_bits4(f32x4 v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);  // a NaN is the largest
  return m;
}
MOE_DEV uint32_t max_over_g(uint32_t m) {  // the four lanes of one token
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  return max(m, (uint32_t)__shfl_xor((int)m, 32));
}

// The FP8 block scale amax / 448 (1 for an all-zero block) and its reciprocal; never below
// the smallest normal number, whose reciprocal is finite.  A NaN maximum is a NaN scale.
MOE_DEV float fp8_scale(uint32_t amax, float& inv) {
  const float s = __uint_as_float(amax) / 448.0f;
  const float sc = amax == 0 ? 1.0f : (s < 1.17549435e-38f ? 1.17549435e-38f : s);
  inv = 1.0f / sc;
  return sc;
}
// Four values of magnitude at most 448 (1 + 2^-22) to E4M3 codes: they round to 448 at most, so
// they need no saturation, and a NaN stays one.
MOE_DEV int e4m3x4(f32x4 v) {
  return __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false), true);
}

// KSP: waves that share one slice of 16 CT columns.  D: K-steps in flight per wave.
// FP8: waves with the whole K quantise the workgroup's 128 columns, the others leave h in fp32.
template <Fmt F, int WAVES, int KSP, int CT, int D>
__global__ __launch_bounds__(64 * WAVES) void few_gate_up_kernel(FewParams p) {
  constexpr int kSlices = WAVES / KSP;
  constexpr bool kBlock = F == Fmt::FP8 && KSP == 1;
  static_assert(!kBlock || WAVES * CT == 8, "the workgroup holds one block");
  static_assert(F != Fmt::MX || CT % 2 == 0, "a wave holds whole blocks of 32 columns");
  __shared__ RouteLds route;
  __shared__ f32x4 red[KSP > 1 ? WAVES : 1][KSP > 1 ? CT * 2 : 1][KSP > 1 ? 64 : 1];
  __shared__ uint32_t amax[kBlock ? WAVES : 1][16];
  const int tid = threadIdx.x, lane = lane_id(), g = lane >> 4, r16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  __shared__ int col[32];  // the columns of this workgroup's expert
  if (blockIdx.y == gridDim.y - 1) {  // the down launch's tables and counters: one workgroup of the last row
    if (blockIdx.x != 0) return;
    __shared__ float tw[kFewMaxPairs];
    __shared__ short ustart[kFewMaxExperts];
    if (p.splits > 1)
      for (int i = tid; i < p.n_blocks; i += 64 * WAVES) p.arrived[i] = 0;
    route_to_lds<WAVES>(p, route, tw);
    write_tables<WAVES>(p, route, tw, ustart);
    return;
  }
  if (tid < 32) col[tid] = 0x7FFF;
  route_to_lds<WAVES>(p, route, nullptr);

  // this workgroup's unit
  const int n_slices = (p.I + 16 * CT - 1) / (16 * CT);
  const int a = (int)blockIdx.y, slice = (int)blockIdx.x * kSlices + wave / KSP;
  int e = -1, half = 0;
  for_units(route, p.E, [&](int before, int le, int n) {
    const uint64_t hit = __ballot(a >= before && a < before + n);
    if (hit == 0) return false;
    const int src = __ffsll((unsigned long long)hit) - 1;
    e = __builtin_amdgcn_readlane(le, src);
    half = a - __builtin_amdgcn_readlane(before, src);
    return true;
  });
  if (e < 0) return;  // (uniform: fewer units than workgroup rows)

  // the columns of the expert: each of its tokens, with the token's first slot of it
  const uint32_t mask = route.mask[e];
  for (int q = tid; q < p.T * p.topk; q += 64 * WAVES)
    if (route.ids[q] == e) {
      const int tq = q / p.topk;
      atomicMin(&col[rank_in(mask, tq)], kCol(tq, q - tq * p.topk));
    }
  __syncthreads();
  const int c = col[16 * half + r16];
  const int t = c == 0x7FFF ? -1 : c >> 5, slot = c & 31;
  // the lane's first byte of a K-step, as XFrag describes
  const uint32_t at = F == Fmt::NV4    ? 128u * (g >> 1) + 16u * (g & 1)
                      : F == Fmt::NVF4 ? 32u * (g >> 1) + 4u * (g & 1)
                                       : 16u * g;
  const uint32_t sat = F == Fmt::MX ? (uint32_t)g : F == Fmt::NVF4 ? 4u * (g >> 1) : 0u;
  const uint32_t xo = t >= 0 ? (uint32_t)t * p.x_row + at : kOOB;
  const uint32_t xso = t >= 0 ? (uint32_t)t * p.x_sf_row + sat : kOOB;
  const __amdgpu_buffer_rsrc_t x_rs = make_rsrc(p.x, (uint32_t)p.T * p.x_row);
  const __amdgpu_buffer_rsrc_t xs_rs = make_rsrc(p.x_sf, (uint32_t)p.T * p.x_sf_row);
  const __amdgpu_buffer_rsrc_t w_rs = make_rsrc(p.w + (size_t)e * p.w_expert, p.w_expert);
  const __amdgpu_buffer_rsrc_t ws_rs = make_rsrc(p.w_sf + (size_t)e * p.w_sf_expert, p.w_sf_expert);
  const bool live = slice < n_slices;
  const int col0 = slice * 16 * CT;
  WAddr<F> wa[CT][2];  // gate, up
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      wa[c][u] = w_addr<F>(slice * CT + c, u, slice * CT + c + u * (p.I / 16), p.ksteps, g, r16,
                           (slice * CT + c) * 16 < p.I);
  // FP8: the 128-row blocks' scales
  const float* sbg = (const float*)(p.w_sf + (size_t)e * p.w_sf_expert) + (size_t)((live ? col0 : 0) / 128) * p.ksteps;
  const float* sbu = sbg + (size_t)(p.I / 128) * p.ksteps;

  struct Stage {
    WFrag<F> w[CT][2];
    XFrag<F, true> x;
    float sg, su;
  } st[D];
  auto load = [&](Stage& s, int k) {
    const uint32_t dead = oob_if(k >= p.steps);
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int u = 0; u < 2; ++u) w_load<F>(s.w[c][u], wa[c][u], w_rs, ws_rs, k, dead, p.ksteps, g);
    if constexpr (F == Fmt::FP8) {
      const int kc = min(k, p.steps - 1);
      s.sg = sbg[kc];
      s.su = sbu[kc];
    }
    const uint32_t o = xo | dead;
    if constexpr (F == Fmt::FP8) {
      s.x.v[0] = bload16(x_rs, o, (uint32_t)k * 128u);
      s.x.v[1] = bload16(x_rs, o + 64u, (uint32_t)k * 128u);
      s.x.s = (int)__builtin_amdgcn_raw_buffer_load_b32(xs_rs, xso | dead, (uint32_t)k * 4u, 0);
    } else if constexpr (F == Fmt::MX) {
      // K tail: rows of any multiple of 32 elements
      s.x.v[0] = bload16(x_rs, o | oob_if(k * 128 + 16 * g >= p.H), (uint32_t)k * 128u);
      s.x.v[1] = bload16(x_rs, (o + 64u) | oob_if(k * 128 + 64 + 16 * g >= p.H), (uint32_t)k * 128u);
      s.x.s = (int)__builtin_amdgcn_raw_buffer_load_b8(xs_rs, xso | dead | oob_if(k * 128 + 32 * g >= p.H),
                                                       (uint32_t)k * 4u, 0);
    } else if constexpr (F == Fmt::BF16) {
      s.x.v[0] = bload16(x_rs, o, (uint32_t)k * 128u);
      s.x.v[1] = bload16(x_rs, o + 64u, (uint32_t)k * 128u);
    } else if constexpr (F == Fmt::NV4) {
      const uint32_t o2 = o | oob_if(2 * k + (g >> 1) >= p.ksteps);
#pragma unroll
      for (int q = 0; q < 4; ++q) s.x.v[q] = bload16(x_rs, o2 + 32u * q, (uint32_t)k * 256u);
    } else {
      const uint32_t odd = oob_if(2 * k + (g >> 1) >= p.ksteps);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        s.x.v[0][q] = (int)__builtin_amdgcn_raw_buffer_load_b32(x_rs, (o | odd) + 8u * q, (uint32_t)k * 64u, 0);
      s.x.s = (int)__builtin_amdgcn_raw_buffer_load_b32(xs_rs, xso | dead | odd, (uint32_t)k * 8u, 0);
    }
  };
  f32x4 acc[CT][2];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int u = 0; u < 2; ++u) acc[c][u] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto mul = [&](const Stage& s) {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if constexpr (F == Fmt::FP8) {
          const float sc = __builtin_bit_cast(float, s.x.s) * (u ? s.su : s.sg);
          const f32x4 part = mma_step<F, true>(s.w[c][u], s.x, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[c][u][i] = fmaf(part[i], sc, acc[c][u][i]);
        } else {
          acc[c][u] = mma_step<F, true>(s.w[c][u], s.x, acc[c][u]);
        }
      }
  };
  int k = wave % KSP;
#pragma unroll
  for (int d = 0; d < D; ++d) load(st[d], k + d * KSP);
  for (; k < p.steps; k += D * KSP) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      mul(st[d]);
      __builtin_amdgcn_sched_barrier(0);
      load(st[d], k + (D + d) * KSP);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // the K parts, in order
  if constexpr (KSP > 1) {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int u = 0; u < 2; ++u) red[wave][c * 2 + u][lane] = acc[c][u];
    __syncthreads();
    if (wave % KSP != 0) return;
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int w = 1; w < KSP; ++w) acc[c][u] += red[wave + w][c * 2 + u][lane];
  }
  if (!live) return;  // (never in a block of FP8: I is a multiple of 128)

  // lane (g, token): columns col0 + 16 c + 4 g ... of the token's row
  const float gs = nv4w(F) ? p.w_gs[e] : 1.0f;
  const size_t row = (size_t)max(t, 0) * p.topk + slot;  // (not used without a token)
  f32x4 h[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    f32x4 gt = acc[c][0], up = acc[c][1];
    if constexpr (nv4w(F)) gt *= gs, up *= gs;
    h[c] = swiglu4(gt, up, p.clamp, p.fast);
  }
  if constexpr (kBlock) {
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < CT; ++c) m = max(m, amax_bits4(h[c]));
    m = max_over_g(m);
    if (g == 0) amax[wave][r16] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) m = max(m, amax[w][r16]);
    float inv;
    const float sc = fp8_scale(m, inv);
    if (t < 0) return;
#pragma unroll
    for (int c = 0; c < CT; ++c) *(int*)((uint8_t*)p.h + row * p.I + col0 + 16 * c + 4 * g) = e4m3x4(h[c] * inv);
    if (wave == 0 && g == 0) ((float*)p.h_sf)[row * (p.I / 128) + col0 / 128] = sc;
  } else if constexpr (F == Fmt::MX) {
#pragma unroll
    for (int b = 0; b < CT; b += 2) {
      const uint32_t m = max_over_g(max(amax_bits4(h[b]), amax_bits4(h[b + 1])));
      const int ex = mx_exponent_for_amax(__uint_as_float(m));
      const float inv = exp2i(-ex);
      const int at = col0 + 16 * b;
      if (t < 0 || at >= p.I) continue;
#pragma unroll
      for (int c = b; c < b + 2; ++c)
        *(uint32_t*)((uint8_t*)p.h + row * p.I + col0 + 16 * c + 4 * g) =
            f32x2_to_e4m3_sat(h[c][0] * inv, h[c][1] * inv) | f32x2_to_e4m3_sat(h[c][2] * inv, h[c][3] * inv) << 16;
      // (a NaN in the block: UE8M0's NaN)
      if (g == 0) ((uint8_t*)p.h_sf)[row * (p.I / 32) + at / 32] = m > 0x7F800000u ? (uint8_t)255 : (uint8_t)(ex + 127);
    }
  } else {
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      f32x4 v = h[c];
      const int at = col0 + 16 * c + 4 * g;
      if constexpr (F == Fmt::NVF4) {
        // block scale E4M3(amax / (6 c)), codes E2M1(h / (scale c)); kept as code x scale, exact in fp16
        const uint32_t m = max_over_g(amax_bits4(v));
        const float cs = p.c_gs[e], s6 = __uint_as_float(m) / (6.0f * cs);
        const float sc = e4m3_byte<0>(__builtin_amdgcn_cvt_pk_fp8_f32(s6 > 448.0f ? 448.0f : s6, 0.0f, 0, false));
        const float den = sc * cs, inv = den > 0.0f ? 1.0f / den : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = e2m1_rne_sat(v[i] * inv) * sc;  // (a NaN in the block: sc is NaN)
      }
      if (t < 0 || at >= p.I) continue;
      if constexpr (F == Fmt::FP8) *(f32x4*)((float*)p.h + row * p.I + at) = v;
      else if constexpr (F == Fmt::NVF4)
        *(uint2*)((uint16_t*)p.h + row * p.I + at) =
            uint2{__builtin_bit_cast(uint32_t, f16x2{(_Float16)v[0], (_Float16)v[1]}),
                  __builtin_bit_cast(uint32_t, f16x2{(_Float16)v[2], (_Float16)v[3]})};
      else *(uint2*)((uint16_t*)p.h + row * p.I + at) = uint2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
    }
  }
}

// A workgroup barrier that waits for this wave's LDS accesses only.
MOE_DEV void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// ---------------------------------------------------------------- down
// R: 16-row weight tiles (output column groups) per workgroup.  HL (FP8): h is fp32 and
// quantised into LDS here.
template <Fmt F, int WAVES, int R, int D, bool HL>
__global__ __launch_bounds__(64 * WAVES) void few_down_kernel(FewParams p) {
  static_assert(!HL || F == Fmt::FP8, "only FP8 leaves h in fp32");
  __shared__ int last;
  extern __shared__ f32x4 sum[];  // [WAVES][R][T][4]: a wave's sums per token and run of 4 rows
  // HL: 128 zero bytes, then the rows' codes (row stride I + 16: rows in other banks); their scales
  __shared__ __attribute__((aligned(16))) uint8_t hq[HL ? 128 + kFewLdsH : 16];
  __shared__ float hsc[HL ? kFewLdsH / 128 : 1];
  const int tid = threadIdx.x, lane = lane_id(), g = lane >> 4, r16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int np = p.T * p.topk;
  // HL: 16 lanes a 128-column block, 8 columns a lane (rows of masked slots hold anything and are not
  // read).  The first kHB chunks of a thread are in flight during the set-up below.
  constexpr int kHB = 4;
  const int cpr = p.I / 8, n_chunks = HL ? np * cpr : 0;
  f32x4 hv[HL ? kHB : 1][2];
  const __amdgpu_buffer_rsrc_t hf_rs = make_rsrc(p.h, (uint32_t)n_chunks * 32u);  // (past the end: zeros)
  auto load_h = [&](int c0) {
    if constexpr (HL) {
#pragma unroll
      for (int i = 0; i < kHB; ++i) {
        const uint32_t o = (uint32_t)(c0 + tid + i * 64 * WAVES) * 32u;
        hv[i][0] = __builtin_bit_cast(f32x4, bload16(hf_rs, o, 0));
        hv[i][1] = __builtin_bit_cast(f32x4, bload16(hf_rs, o + 16u, 0));
      }
    }
  };
  auto quantise_h = [&](int c0) {
    if constexpr (HL) {
#pragma unroll
      for (int i = 0; i < kHB; ++i) {
        const int c = c0 + tid + i * 64 * WAVES;
        uint32_t m = max(amax_bits4(hv[i][0]), amax_bits4(hv[i][1]));
        m = dpp_max_u32<0xB1>(m);
        m = dpp_max_u32<0x4E>(m);
        m = dpp_max_u32<0x141>(m);
        m = dpp_max_u32<0x140>(m);
        float inv;
        const float sc = fp8_scale(m, inv);
        if (c < n_chunks) {
          const int row = c / cpr, col = c - row * cpr;
          *(uint2*)(hq + 128 + row * (p.I + 16) + col * 8) =
              uint2{(uint32_t)e4m3x4(hv[i][0] * inv), (uint32_t)e4m3x4(hv[i][1] * inv)};
          if ((lane & 15) == 0) hsc[c >> 4] = sc;
        }
      }
    }
  };
  load_h(0);
  const int entries = R * p.T * 4;
  for (int i = lane; i < entries; i += 64) sum[wave * entries + i] = f32x4{0.f, 0.f, 0.f, 0.f};
  // the units' tables
  uint32_t* tables = (uint32_t*)(sum + WAVES * entries);
  const FewTables tb = few_tables(tables, np, p.max_units);
  for (int i = tid; i < (int)few_table_words(np, p.max_units); i += 64 * WAVES) tables[i] = p.tables[i];
  const int n_units = (int)*p.tables;
  __syncthreads();

  // this wave's part of the (unit, K-step) sequence
  const int blk = (int)blockIdx.x, split = (int)blockIdx.y;
  const uint32_t total = (uint32_t)n_units * (uint32_t)p.steps;
  const int at = split * WAVES + wave;
  const int share = (int)(p.splits == 1 ? total / WAVES : total / (uint32_t)(p.splits * WAVES));
  const int more = (int)total - share * p.splits * WAVES;  // parts of one step more
  const int lo = at * share + min(at, more), hi = lo + share + (at < more ? 1 : 0);
  const int rb0 = blk * R;  // first 16-row block
  const int n_rb = p.H / 16;
  WAddr<F> wa[R];
#pragma unroll
  for (int r = 0; r < R; ++r) wa[r] = w_addr<F>((rb0 + r) >> 1, (rb0 + r) & 1, rb0 + r, p.ksteps, g, r16, rb0 + r < n_rb);

  const uint32_t h_row = HL ? (uint32_t)p.I + 16u : (uint32_t)p.I * (mma16(F) ? 2u : 1u);
  const uint32_t hs_row = F == Fmt::FP8 ? (uint32_t)(p.I / 128) * (HL ? 1u : 4u) : (uint32_t)(p.I / 32);
  const uint32_t rows = (uint32_t)(p.T * p.topk);
  const __amdgpu_buffer_rsrc_t h_rs = make_rsrc(p.h, rows * h_row);
  const __amdgpu_buffer_rsrc_t hs_rs = make_rsrc(p.h_sf, rows * hs_row);

  // the load side's position: unit, its expert's resources, the lane's token, row and router weight
  int lu = (int)((uint32_t)lo / (uint32_t)p.steps), lk = lo - lu * p.steps, lf = lo;
  __amdgpu_buffer_rsrc_t w_rs, ws_rs;
  const float* sb = nullptr;
  uint32_t ho, hso;
  float wt;
  int tok;
  auto set_unit = [&]() {
    const int lc = max(min(lu, n_units - 1), 0);
    const int u = __builtin_amdgcn_readfirstlane((int)tb.unit[lc]), e = u & 0xFFFF;
    const int c = ((const unsigned short*)tb.col)[lc * 16 + r16];
    w_rs = make_rsrc(p.w + (size_t)e * p.w_expert, p.w_expert);
    ws_rs = make_rsrc(p.w_sf + (size_t)e * p.w_sf_expert, p.w_sf_expert);
    if constexpr (F == Fmt::FP8)
      sb = (const float*)(p.w_sf + (size_t)e * p.w_sf_expert) + (size_t)(rb0 / 8) * p.ksteps;
    const bool mine = r16 < u >> 16;
    tok = mine ? c >> 5 : -1;
    const uint32_t row = mine ? (uint32_t)((c >> 5) * p.topk + (c & 31)) : 0u;
    wt = __builtin_bit_cast(float, tb.w[row]);
    if constexpr (nv4w(F)) wt *= p.w_gs[e];
    const uint32_t at = nv4w(F) ? 128u * (g >> 1) + 16u * (g & 1) : 16u * g;
    ho = tok >= 0 ? row * h_row + at : kOOB;
    hso = tok >= 0 ? row * hs_row + (F == Fmt::MX ? (uint32_t)g : 0u) : kOOB;
  };
  struct Stage {
    WFrag<F> w[R];
    XFrag<F, false> x;
    float wt, sb;
    uint32_t off, soff;  // HL: the row's place in LDS
    int k, tok;
    bool last;  // of the unit, or of the wave's part
  } st[D];
  auto load = [&](Stage& s) {
    const uint32_t dead = oob_if(lf >= hi);
    const int k = lk;
#pragma unroll
    for (int r = 0; r < R; ++r) w_load<F>(s.w[r], wa[r], w_rs, ws_rs, k, dead, p.ksteps, g);
    if constexpr (F == Fmt::FP8) s.sb = sb[k];
    const uint32_t o = ho | dead;
    s.wt = wt;
    s.tok = tok;
    if constexpr (HL) {
      s.off = ho;
      s.soff = hso;
      s.k = k;
    } else if constexpr (F == Fmt::FP8) {
      s.x.v[0] = bload16(h_rs, o, (uint32_t)k * 128u);
      s.x.v[1] = bload16(h_rs, o + 64u, (uint32_t)k * 128u);
      s.x.s = (int)__builtin_amdgcn_raw_buffer_load_b32(hs_rs, hso | dead, (uint32_t)k * 4u, 0);
    } else if constexpr (F == Fmt::MX) {
      s.x.v[0] = bload16(h_rs, o | oob_if(k * 128 + 16 * g >= p.I), (uint32_t)k * 128u);
      s.x.v[1] = bload16(h_rs, (o + 64u) | oob_if(k * 128 + 64 + 16 * g >= p.I), (uint32_t)k * 128u);
      s.x.s = (int)__builtin_amdgcn_raw_buffer_load_b8(hs_rs, hso | dead | oob_if(k * 128 + 32 * g >= p.I),
                                                       (uint32_t)k * 4u, 0);
    } else if constexpr (F == Fmt::BF16) {
      s.x.v[0] = bload16(h_rs, o, (uint32_t)k * 128u);
      s.x.v[1] = bload16(h_rs, o + 64u, (uint32_t)k * 128u);
    } else {
      const uint32_t o2 = o | oob_if(2 * k + (g >> 1) >= p.ksteps);
#pragma unroll
      for (int q = 0; q < 4; ++q) s.x.v[q] = bload16(h_rs, o2 + 32u * q, (uint32_t)k * 256u);
    }
    s.last = lf < hi && (lk + 1 == p.steps || lf + 1 == hi);
    ++lf;
    if (++lk == p.steps) {  // (uniform)
      lk = 0;
      ++lu;
      set_unit();
    }
  };
  f32x4 acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto mul = [&](Stage& s) {
    float c = s.wt;
    if constexpr (HL) {
      const bool ok = s.tok >= 0;
      const uint32_t at = ok ? 128u + s.off + (uint32_t)s.k * 128u : 16u * g;
      s.x.v[0] = *(const i32x4*)(hq + at);
      s.x.v[1] = *(const i32x4*)(hq + at + 64);
      c *= hsc[ok ? s.soff + (uint32_t)s.k : 0u] * s.sb;
    } else if constexpr (F == Fmt::FP8) {
      c *= __builtin_bit_cast(float, s.x.s) * s.sb;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // FP8: each K-step's partial has its own scales; the others scale the unit's sum
      if constexpr (F == Fmt::FP8) {
        const f32x4 part = mma_step<F, false>(s.w[r], s.x, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][i] = fmaf(part[i], c, acc[r][i]);
      } else {
        acc[r] = mma_step<F, false>(s.w[r], s.x, acc[r]);
      }
    }
    if (s.last) {  // (uniform)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (s.tok >= 0) {
          f32x4& at = sum[wave * entries + (r * p.T + s.tok) * 4 + g];
          f32x4 v = at;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = F == Fmt::FP8 ? v[i] + acc[r][i] : fmaf(acc[r][i], c, v[i]);
          at = v;
        }
        acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
  };
  const bool busy = lo < hi;  // (uniform per wave)
  if (busy) {
    set_unit();
#pragma unroll
    for (int d = 0; d < D; ++d) load(st[d]);
  }
  if constexpr (HL) {
    if (tid < 32) ((uint32_t*)hq)[tid] = 0;
    quantise_h(0);
    for (int c0 = kHB * 64 * WAVES; c0 < n_chunks; c0 += kHB * 64 * WAVES) {
      load_h(c0);
      quantise_h(c0);
    }
    lds_barrier();  // (the weights stay in flight)
  }
  if (busy) {
    for (int f = lo; f < hi; f += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        mul(st[d]);
        __builtin_amdgcn_sched_barrier(0);
        load(st[d]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  __syncthreads();
  auto wave_sum = [&](int i) {
    f32x4 v = sum[i];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += sum[w * entries + i];
    return v;
  };
  auto finish = [&](int i, f32x4 v) {
    const int t = (i >> 2) % p.T, rb = rb0 + i / (p.T * 4);
    if (rb >= n_rb) return;
    const size_t at = (size_t)t * p.H + 16 * rb + 4 * (i & 3);
    const uint16_t* add[2] = {p.shared, p.residual};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (add[q] == nullptr) continue;
      const uint2 a = *(const uint2*)(add[q] + at);
      v += f32x4{__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xFFFF0000u), __uint_as_float(a.y << 16),
                 __uint_as_float(a.y & 0xFFFF0000u)};
    }
    if (p.out_f32) *(f32x4*)((float*)p.out + at) = v;
    else *(uint2*)((uint16_t*)p.out + at) = uint2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
  };
  if (p.splits == 1) {
    for (int i = tid; i < entries; i += 64 * WAVES) finish(i, wave_sum(i));
    return;
  }
  // Device-scope stores, completed before the workgroup arrives; device-scope loads by the last one.
  // No waiting, no data atomics.
  const __amdgpu_buffer_rsrc_t p_rs = make_rsrc(p.part, (uint32_t)(p.splits * p.n_blocks * entries) * 16u);
  for (int i = tid; i < entries; i += 64 * WAVES)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, wave_sum(i)), p_rs,
                                           (uint32_t)((split * p.n_blocks + blk) * entries + i) * 16u, 0, kCpolDevice);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (tid == 0) last = atomicAdd(p.arrived + blk, 1) == p.splits - 1;
  __syncthreads();
  if (!last) return;
  for (int i = tid; i < entries; i += 64 * WAVES) {
    f32x4 v[kFewMaxSplits];
#pragma unroll
    for (int q = 0; q < kFewMaxSplits; ++q) {  // (all in flight at once; past the last split: zeros)
      const uint32_t o = q < p.splits ? (uint32_t)((q * p.n_blocks + blk) * entries + i) * 16u : kOOB;
      v[q] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(p_rs, o, 0, kCpolDevice));
    }
#pragma unroll
    for (int q = 1; q < kFewMaxSplits; ++q) v[0] += v[q];
    finish(i, v[0]);
  }
}

}  // namespace

// The top-k in the first launch saves a launch, but every workgroup repeats it.  Measured, us, in the
// launch / before it: MX H 2880, I 2880, E 128, k 4: T 1 20.7 / 22.2, T 4 48.3 / 48.6, T 8 80.8 / 71.7,
// T 32 381 / 177; FP8 H 7168, I 256, E 256, k 8: T 1 22.4 / 23.7, T 4 38.6 / 40.2, T 8 68.3 / 64.5.
bool few_routes_in_launch(int T) { return T <= 4; }

// FP8: h in fp32 between the launches (see above).  Whole 128-column blocks need about as many
// workgroups as the part has CUs to stream at full rate.  Measured, us for the layer, fp32 h / blocks:
// T 1, H 7168, I 2048, k 8 62.0 / 74.5; I 256 17.3 / 45.9; T 5, H 256, I 128 9.9 / 10.9.
static bool few_h_fp32(Fmt f, int T, int topk, int E, int I) {
  const int pairs = T * topk, active = min(E, pairs);
  return f == Fmt::FP8 && (long long)active * (I / 128) < 256 && (long long)pairs * (I + 16) <= kFewLdsH;
}
// The down launch's blocks: 16 rows per wave's weight tile, tiles per workgroup, splits: as many as
// leave no CU a second workgroup.  Measured, us for the layer, MX, T 32, H 2880, I 2880, E 128, k 4
// (45 blocks of 4 tiles): 1 split 324, 4 196, 5 (225 workgroups) 188, 6 216, 8 201; 2 tiles in 4 splits 207.
// FP8, T 16, H 7168, I 2048: 224 blocks of 2 tiles 220, 448 of 1 tile 232.  BF16, T 4, H 4096,
// I 14336: 256 blocks of 1 tile 250, 128 of 2 tiles in 2 splits 275.
struct DownPlan {
  int rows, n_blocks, splits;
};
// Twice the tiles where that fills more of the part and a wave has more than four K-steps (BF16, T 10, H 5248,
// I 768: 328 blocks of 1 tile 50.0, 164 of 2 46.2; FP8, T 16, H 4224, I 1024: 132 of 2 56.8, 66 of 4 in 3 splits
// 53.2; NVFP4, T 20, H 2880, I 2880: 90 in 2 splits 99, 45 in 5 92.  At equal counts: BF16, H 4096 248 and 251;
// with short parts: FP8, T 2, H 4224, I 512 16.8 and 18.0.)
static DownPlan down_plan_rows(int H, int rows) {
  const int n = (H / 16 + rows - 1) / rows;
  return DownPlan{rows, n, max(1, min(256 / n, kFewMaxSplits))};
}
static DownPlan down_plan(Fmt f, int H, long long steps) {  // steps: K-steps of all units
  auto used = [](const DownPlan& d) { return d.n_blocks > 256 ? 0 : d.n_blocks * d.splits; };  // of one round
  const DownPlan few = down_plan_rows(H, f == Fmt::BF16 ? 1 : f == Fmt::MX ? 4 : 2);
  const DownPlan many = down_plan_rows(H, 2 * few.rows);
  return f != Fmt::MX && used(many) > used(few) && steps > 4LL * many.splits * 8 ? many : few;
}
FewBuffers few_buffers(Fmt f, int T, int topk, int E, int H, int I) {
  FewBuffers b{};
  if (T == 0) return b;
  const size_t pairs = (size_t)T * topk;
  // (FP8: room for fp32 whether this T takes it or not, so that the size never shrinks as T grows)
  b.h = pairs * I * (f == Fmt::FP8 ? 4 : mma16(f) ? 2 : 1);
  b.h_sf = f == Fmt::FP8 ? pairs * (I / 128) * 4 : f == Fmt::MX ? pairs * (I / 32) : 0;
  b.tables = few_table_words(T * topk, few_max_units(E, T, topk)) * 4;
  for (const long long steps : {0LL, 1LL << 40}) {  // either plan
    const DownPlan d = down_plan(f, H, steps);
    if (d.splits == 1) continue;
    b.arrived = std::max(b.arrived, (size_t)d.n_blocks * 4);
    b.part = std::max(b.part, (size_t)d.splits * d.n_blocks * d.rows * T * 64);
  }
  return b;
}

hipError_t launch_few(const FewArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  const Fmt wf = a.fmt == Fmt::NVF4 ? Fmt::NV4 : a.fmt;
  FewParams p{};
  p.T = a.T;
  p.topk = a.topk;
  p.E = a.E;
  p.H = a.H;
  p.I = a.I;
  p.fast = a.fast ? 1 : 0;
  p.clamp = a.clamp;
  p.ids = a.ids;
  p.ids64 = a.ids64 ? 1 : 0;
  p.topk_w = a.topk_w;
  p.h = a.h;
  p.h_sf = a.h_sf;
  p.shared = (const uint16_t*)a.shared;
  p.residual = (const uint16_t*)a.residual;
  p.out = a.out;
  p.out_f32 = a.out_f32 ? 1 : 0;

  const long long units = min(a.E, a.T * a.topk);
  const int ksteps = prepared_ksteps(wf, a.I), steps = nv4w(a.fmt) ? (ksteps + 1) / 2 : ksteps;  // the down leg's
  const DownPlan dp = down_plan(a.fmt, a.H, units * steps);
  p.splits = dp.splits;
  p.n_blocks = dp.n_blocks;
  p.tables = (uint32_t*)a.tables;
  p.max_units = few_max_units(a.E, a.T, a.topk);
  p.arrived = (int*)a.arrived;
  p.part = (float*)a.part;

  FewParams u = p;  // gate_up
  u.logits = a.logits;
  u.bias = a.bias;
  if (a.logits != nullptr) {
    if (a.ids64) u.idx64_out = (long long*)a.ids;
    else u.idx32_out = (int*)a.ids;
    u.w_out = (float*)a.topk_w;
  }
  u.x = (const uint8_t*)a.x;
  u.x_sf = (const uint8_t*)a.x_sf;
  u.x_row = a.fmt == Fmt::NVF4 ? a.H / 2 : mma16(a.fmt) ? 2 * a.H : a.H;
  u.x_sf_row = a.fmt == Fmt::FP8 ? a.H / 128 * 4 : a.fmt == Fmt::MX ? a.H / 32 : a.fmt == Fmt::NVF4 ? a.H / 16 : 0;
  u.w = (const uint8_t*)a.w13;
  u.w_sf = (const uint8_t*)a.w13_sf;
  u.w_expert = (uint32_t)prepared_expert_bytes(wf, 2 * a.I, a.H);
  u.w_sf_expert = a.fmt == Fmt::FP8 ? (uint32_t)(2 * a.I / 128 * (a.H / 128) * 4)
                                    : (uint32_t)prepared_scale_expert_bytes(wf, 2 * a.I, a.H);
  u.w_gs = a.w13_gs;
  u.c_gs = a.c_scales;
  u.ksteps = prepared_ksteps(wf, a.H);
  u.steps = nv4w(a.fmt) ? (u.ksteps + 1) / 2 : u.ksteps;

  FewParams d = p;  // down
  d.w = (const uint8_t*)a.w2;
  d.w_sf = (const uint8_t*)a.w2_sf;
  d.w_expert = (uint32_t)prepared_expert_bytes(wf, a.H, a.I);
  d.w_sf_expert = a.fmt == Fmt::FP8 ? (uint32_t)(a.H / 128 * (a.I / 128) * 4)
                                    : (uint32_t)prepared_scale_expert_bytes(wf, a.H, a.I);
  d.w_gs = a.w2_gs;
  d.ksteps = ksteps;
  d.steps = steps;

  auto up = [&](auto fmt, auto waves, auto ksp, auto groups, auto depth) {
    constexpr Fmt F = decltype(fmt)::value;
    constexpr int W = decltype(waves)::value, KSP = decltype(ksp)::value, CT = decltype(groups)::value,
                  D = decltype(depth)::value;
    constexpr int per = W / KSP * 16 * CT;  // columns of h per workgroup
    const dim3 grid((unsigned)((a.I + per - 1) / per), (unsigned)(p.max_units + 1));
    hipLaunchKernelGGL((few_gate_up_kernel<F, W, KSP, CT, D>), grid, dim3(64 * W), 0, s, u);
  };
  auto down = [&](auto fmt, auto waves, auto rows, auto depth, auto lds_h) {
    constexpr Fmt F = decltype(fmt)::value;
    constexpr int W = decltype(waves)::value, R = decltype(rows)::value, D = decltype(depth)::value;
    const size_t lds = (size_t)W * R * a.T * 64 + few_table_words(a.T * a.topk, p.max_units) * 4;
    hipLaunchKernelGGL((few_down_kernel<F, W, R, D, decltype(lds_h)::value>), dim3((unsigned)dp.n_blocks, (unsigned)dp.splits),
                       dim3(64 * W), lds, s, d);
  };
  // The waves of gate_up share a slice's K-steps by four: BF16, T 4, H 4096, I 14336 248 us, by two 254, whole
  // 266 (T 1, H 2048, I 1024: 18.1, 21.1, 25.6; FP8, T 1, a 1/8 shard: 18.4 by four, 23.6 by two).  By eight, one
  // K-step in flight each, in a single round of workgroups (FP8, T 1, H 7168, I 256: 17.6 against 18.5; MX, T 27,
  // H 4608, I 224, 20 experts: 17.2 against 18.7), not beyond (MX, T 32, I 2880, 128 experts: 202 against 188).
  // MX needs slices of 32 columns (64: T 32 186 against 188 us, T 1 24.1 against 22.8) and keeps one K-step in
  // flight per wave (T 32 182, two 187); FP8 and BF16 two (T 16 216, one 225; T 4 248 and 249).  NVFP4's x operand serves
  // two slices of 16 where they still make a round: T 20, H 2880, I 2880 100 us against 110, T 16, H 7168, I 2048
  // 151 against 162; not with fewer: T 1, H 7168, I 256 25.9 against 18.9 (by eight 17.0).
  const bool wide = units * ((a.I + 31) / 32) >= 256;
  const bool thin = units * ((a.I + 31) / 32) * (a.fmt == Fmt::MX ? 1 : 2) <= 256;
  // down: K-steps in flight per wave.  One: FP8, T 16, H 7168, I 2048 216 us, two 220; MX, T 1, H 2880, I 2880
  // 22.2 and 23.1.  Two: BF16, T 4, H 4096, I 14336 248, one 262; NVFP4, T 20, H 2880, I 2880 99 and 107, unless a
  // wave has only a step or two (T 1, H 2048, I 1024 13.8, one 13.0).
  const bool brief = units * steps <= 2LL * dp.splits * 8;
#define C_(v) std::integral_constant<int, v>{}
#define F_(v) std::integral_constant<Fmt, v>{}
  switch (a.fmt) {
    case Fmt::FP8:
      if (few_h_fp32(a.fmt, a.T, a.topk, a.E, a.I)) {
        if (thin) up(F_(Fmt::FP8), C_(8), C_(8), C_(1), C_(1));
        else up(F_(Fmt::FP8), C_(4), C_(4), C_(1), C_(2));
        if (dp.rows == 2) down(F_(Fmt::FP8), C_(8), C_(2), C_(1), std::true_type{});
        else down(F_(Fmt::FP8), C_(8), C_(4), C_(1), std::true_type{});
      } else {
        up(F_(Fmt::FP8), C_(8), C_(1), C_(1), C_(2));
        if (dp.rows == 2) down(F_(Fmt::FP8), C_(8), C_(2), C_(1), std::false_type{});
        else down(F_(Fmt::FP8), C_(8), C_(4), C_(1), std::false_type{});
      }
      break;
    case Fmt::BF16:
      if (thin) up(F_(Fmt::BF16), C_(8), C_(8), C_(1), C_(1));
      else up(F_(Fmt::BF16), C_(4), C_(4), C_(1), C_(2));
      if (dp.rows == 1) down(F_(Fmt::BF16), C_(8), C_(1), C_(2), std::false_type{});
      else down(F_(Fmt::BF16), C_(8), C_(2), C_(1), std::false_type{});
      break;
    case Fmt::MX:
      if (thin) up(F_(Fmt::MX), C_(8), C_(8), C_(2), C_(1));
      else up(F_(Fmt::MX), C_(4), C_(4), C_(2), C_(1));
      down(F_(Fmt::MX), C_(8), C_(4), C_(1), std::false_type{});
      break;
    case Fmt::NV4:
      if (wide) up(F_(Fmt::NV4), C_(4), C_(4), C_(2), C_(1));
      else up(F_(Fmt::NV4), C_(8), C_(8), C_(1), C_(1));
      if (dp.rows == 4) down(F_(Fmt::NV4), C_(8), C_(4), C_(2), std::false_type{});
      else if (brief) down(F_(Fmt::NV4), C_(8), C_(2), C_(1), std::false_type{});
      else down(F_(Fmt::NV4), C_(8), C_(2), C_(2), std::false_type{});
      break;
    case Fmt::NVF4:
      if (wide) up(F_(Fmt::NVF4), C_(4), C_(4), C_(2), C_(1));
      else up(F_(Fmt::NVF4), C_(8), C_(8), C_(1), C_(1));
      if (dp.rows == 4) down(F_(Fmt::NVF4), C_(8), C_(4), C_(2), std::false_type{});
      else if (brief) down(F_(Fmt::NVF4), C_(8), C_(2), C_(1), std::false_type{});
      else down(F_(Fmt::NVF4), C_(8), C_(2), C_(2), std::false_type{});
      break;
  }
#undef C_
#undef F_
  return hipGetLastError();
}

}  // namespace moe
