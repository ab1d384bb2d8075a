// Router logits: logits[t, e] = sum over h of x[t, h] * W[e, h], x bf16 and W bf16
// or fp32, fp32 sums: what FromLogits routing (the routing_input_mode entry of the
// MoEActivationPack page) starts from.
//
// v_mfma_f32_16x16x32_bf16 with the router's rows as the first operand and the
// tokens as the second.  fp32 weights are split into three bf16 terms whose sum
// holds all 24 bits of the weight (w = w0 + w1 + w2 exactly, barring underflow),
// each multiplied on the matrix cores: bf16 products are exact in fp32, so the
// result has the error of an fp32 sum.
//
// Bound by what one CU can read: on average 87 requests of 128 bytes are in flight in its vector cache, at 550 cycles
// each with x from HBM (49 GB/s; T 8192, H 7168, E 256: 192 lines a K-step and workgroup, 56 us, 540 TFLOP/s), and
// at 58 to 78 GB/s where the operands come from L2 (T 256: 458 KB per 16 x 16 tile, 8.0 us).  fp32 weights: by the
// VALU work of their split.
#include <algorithm>
#include <type_traits>

#include "gemm_common.h"
#include "layer.h"
#include "topk.h"

namespace moe {

namespace {

struct RouterParams {
  const uint8_t* x;
  const uint8_t* w;
  float* out;  // logits, or the partial sums [splits][T][E]
  int T, H, E;
  int n_tiles;   // expert tiles
  int steps;     // K-steps of 64
  int splits;    // workgroups that share a tile's K-steps
};

// Three bf16 terms of 8 fp32 values: the upper half of each word, then of what that
// leaves, then the rest (24 significand bits are 3 x 8, so nothing is lost).  An infinite
// or NaN weight leaves a NaN, as an infinite x does against a term of zero: outputs that
// are NaN are computed again by plain_dot.  (A test of every weight instead: T 512, H 7168,
// E 256 30.1 us, this 25.7.)
MOE_DEV uint32_t high_halves(float lo, float hi) {  // (bf16 of lo, bf16 of hi), truncated
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
MOE_DEV float high_half(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }
MOE_DEV void split3(const f32x4 a, const f32x4 b, i32x4 (&o)[3]) {
  const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float r[2], s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r[i] = v[2 * q + i] - high_half(v[2 * q + i]);
      s[i] = r[i] - high_half(r[i]);
    }
    o[0][q] = (int)high_halves(v[2 * q], v[2 * q + 1]);
    o[1][q] = (int)high_halves(r[0], r[1]);
    o[2][q] = (int)high_halves(s[0], s[1]);
  }
}

// logits[t, e] of fp32 weights without the split (rare: its result was NaN).  A NaN sum is final.  One lane an
// output, so slow: T 8192, H 7168, E 256, one token with a NaN in its last column 125 -> 1920 us, in its first 116.
MOE_DEV float plain_dot(const RouterParams& p, int t, int e) {
  const uint16_t* x = (const uint16_t*)p.x + (size_t)t * p.H;
  const float* w = (const float*)p.w + (size_t)e * p.H;
  float s = 0.0f;
  for (int c = 0; c < p.H && s == s; c += 8) {
    const i32x4 a = *(const i32x4*)(x + c);
    const f32x4 b[2] = {*(const f32x4*)(w + c), *(const f32x4*)(w + c + 4)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s = fmaf(__uint_as_float((uint32_t)a[i] << 16), b[i >> 1][2 * (i & 1)], s);
      s = fmaf(__uint_as_float((uint32_t)a[i] & 0xFFFF0000u), b[i >> 1][2 * (i & 1) + 1], s);
    }
  }
  return s;
}

// ---------------------------------------------------------------- few tokens
// A workgroup per expert, TT >= T tokens: dot products in fp32 on rows read
// in whole lines by all four waves.
template <int TT, bool W32>
__global__ __launch_bounds__(256) void router_dot_kernel(RouterParams p) {
  __shared__ float part[4][TT];
  const int tid = threadIdx.x, e = blockIdx.x, C = p.H >> 3;
  float acc[TT] = {};
  for (int c = tid; c < C; c += 256) {
    float w[8];
    if constexpr (W32) {
      const f32x4* q = (const f32x4*)((const float*)p.w + (size_t)e * p.H + c * 8);
      const f32x4 a = q[0], b = q[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = a[i], w[4 + i] = b[i];
    } else {
      const i32x4 a = *(const i32x4*)((const uint16_t*)p.w + (size_t)e * p.H + c * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[2 * i] = __uint_as_float((uint32_t)a[i] << 16);
        w[2 * i + 1] = __uint_as_float((uint32_t)a[i] & 0xFFFF0000u);
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      // (past the last token: the last one again, not stored)
      const i32x4 x = *(const i32x4*)((const uint16_t*)p.x + (size_t)min(t, p.T - 1) * p.H + c * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[t] = fmaf(__uint_as_float((uint32_t)x[i] << 16), w[2 * i], acc[t]);
        acc[t] = fmaf(__uint_as_float((uint32_t)x[i] & 0xFFFF0000u), w[2 * i + 1], acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const float s = wave_sum_f32(acc[t]);
    if ((tid & 63) == 0) part[tid >> 6][t] = s;
  }
  __syncthreads();
  if (tid < TT && tid < p.T)
    p.out[(size_t)tid * p.E + e] = part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid];
}

// ---------------------------------------------------------------- tiles
// A workgroup computes BM tokens x BN experts.  Rows of x and W are staged in LDS by
// direct-to-LDS loads of whole 128-byte lines (8 lanes a line: MFMA-order loads straight
// into registers put every lane of a quarter wave on another line and ran at 17 bytes per
// cycle and CU), 16-byte chunks XOR-swizzled by row, K-step 64, STG buffers.
// WT waves share a stage, each its part of the tile (1: a wave on its own, no
// barriers); WK such groups, and the workgroups of a split, take the K-steps in
// turn, and their sums are added in order.
template <int BM, int BN, int WT, int WK, int STG, bool W32>
struct RouterTile {
  static constexpr int kF = W32 ? 2 : 1;
  static constexpr int kXBytes = BM * 128, kStage = kXBytes + BN * 128 * kF;
  static constexpr int kThreads = 64 * WT * WK;
  static constexpr int kLds = WK * STG * kStage;
  static constexpr int kLoads = (BM * 8 + BN * 8 * kF) / (64 * WT);  // per lane and stage
};
// (rows r and r + 16 of a 32-row operand are read together: they take different chunks too)
template <int B>
MOE_HOST_DEV constexpr int router_swz(int r) {
  return (r & 7) ^ (B >= 32 ? (r >> 4) & 1 : 0);
}

template <int BM, int BN, int WT, int WK, int STG, bool W32>
__global__ __launch_bounds__(64 * WT * WK) void router_tile_kernel(RouterParams p) {
  using TL = RouterTile<BM, BN, WT, WK, STG, W32>;
  constexpr int F = TL::kF;
  constexpr bool k32 = BM >= 32;           // 32x32x16 MFMA, else 16x16x32
  // Waves over the tile.  fp32 weights: every wave takes all BM tokens, so that each weight is
  // split once (128 x 128 tiles at T 8192, H 7168, E 256, 2 splits: 133 us with 2 x 2 waves, this 112).
  constexpr int WM = WT >= 4 && !W32 ? 2 : 1, WN = WT / WM;
  constexpr int R = k32 ? 32 : 16;
  constexpr int MT = BM / WM / R, NT = BN / WN / R;
  __shared__ __attribute__((aligned(16))) uint8_t lds[TL::kLds];
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = wave / WT, wt = wave % WT, gl = wt * 64 + lane;  // K group, wave and lane of it
  // 16 x 16 tiles: a grid of two axes, no division on the way to the first load (with two: T 128, H 2880, E 128
  // 4.4 us, this 4.15).
  // Larger ones: neighbouring tiles, which share rows of x, on one XCD's L2.
  constexpr bool kSplit = W32 && BM == 128 && BN == 64;  // (the only ones that split K)
  const int splits = kSplit ? p.splits : 1;
  const int id = BM > 16 ? xcd_remap(blockIdx.x, gridDim.x) : 0;
  const int tile = kSplit ? id / splits : id, split = kSplit ? id - tile * splits : 0;
  const int tm = BM > 16 ? tile / p.n_tiles : (int)blockIdx.y, te = BM > 16 ? tile - tm * p.n_tiles : (int)blockIdx.x;
  const int t0 = tm * BM, e0 = te * BN;
  const uint32_t xrow = (uint32_t)p.H * 2, wrow = (uint32_t)p.H * 2 * F;
  // rows past the last one lie past the resource: zeros
  const __amdgpu_buffer_rsrc_t x_rs = make_rsrc(p.x + (size_t)t0 * xrow, (uint32_t)min(BM, p.T - t0) * xrow);
  const __amdgpu_buffer_rsrc_t w_rs = make_rsrc(p.w + (size_t)e0 * wrow, (uint32_t)min(BN, p.E - e0) * wrow);
  uint8_t* mine = lds + kg * STG * TL::kStage;

  auto issue = [&](int k, int buf) {
    const uint32_t dead = oob_if(k >= p.steps);
    const bool half = k * 64 + 32 >= p.H;  // H is a multiple of 32: the last K-step may hold 32 elements
    uint8_t* base = mine + buf * TL::kStage;
#pragma unroll
    for (int i = 0; i < BM * 8 / (64 * WT); ++i) {
      const int s = i * 64 * WT + gl, row = s >> 3, c = (s & 7) ^ router_swz<BM>(row);
      lds_load16(x_rs, base + (i * 64 * WT + wt * 64) * 16, ((uint32_t)row * xrow + 16u * c) | dead | oob_if(half && c >= 4),
                 (uint32_t)k * 128u);
    }
#pragma unroll
    for (int i = 0; i < BN * 8 * F / (64 * WT); ++i) {
      const int s = i * 64 * WT + gl, row = s / (8 * F), q = s % (8 * F), c = (q & 8) | ((q & 7) ^ router_swz<BN>(row));
      lds_load16(w_rs, base + TL::kXBytes + (i * 64 * WT + wt * 64) * 16,
                 ((uint32_t)row * wrow + 16u * c) | dead | oob_if(half && c >= 4 * F), (uint32_t)k * 128u * F);
    }
  };
  typedef float accv __attribute__((ext_vector_type(k32 ? 16 : 4)));
  accv acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = accv{};
  const int r = lane % R, g = lane / R;  // operand row, K group of the lane
  const int m0 = wt / WN * (BM / WM), n0 = wt % WN * (BN / WN);
  auto mul = [&](int buf) {
    const uint8_t* xb = mine + buf * TL::kStage;
    const uint8_t* wb = xb + TL::kXBytes;
    constexpr int kSub = k32 ? 4 : 2, kG = k32 ? 2 : 4;  // MFMAs of a K-step, lanes of a row
#pragma unroll
    for (int sub = 0; sub < kSub; ++sub) {
      const int c = kG * sub + g;  // the lane's 8 elements
      i32x4 xf[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int row = m0 + m * R + r;
        xf[m] = *(const i32x4*)(xb + row * 128 + ((c ^ router_swz<BM>(row)) << 4));
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = n0 + n * R + r, sw = router_swz<BN>(row);
        i32x4 wf[W32 ? 3 : 1];
        if constexpr (W32) {
          const int c0 = 2 * c, c1 = 2 * c + 1;
          const uint8_t* at = wb + row * 256;
          split3(*(const f32x4*)(at + (((c0 & 8) | ((c0 & 7) ^ sw)) << 4)),
                 *(const f32x4*)(at + (((c1 & 8) | ((c1 & 7) ^ sw)) << 4)), wf);
        } else {
          wf[0] = *(const i32x4*)(wb + row * 128 + ((c ^ sw) << 4));
        }
#pragma unroll
        for (int q = (W32 ? 2 : 0); q >= 0; --q)  // the smallest term first
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const bf16x8 a = __builtin_bit_cast(bf16x8, wf[q]), b = __builtin_bit_cast(bf16x8, xf[m]);
            if constexpr (k32) acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[m][n], 0, 0, 0);
            else acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc[m][n], 0, 0, 0);
          }
      }
    }
  };
  const int stride = WK * splits;
  int k = split * WK + kg;
#pragma unroll
  for (int s = 0; s < STG - 1; ++s) issue(k + s * stride, s);
  // Every wave of the workgroup runs the same number of trips.  A stage's loads have landed when
  // only those of the STG - 2 later stages are outstanding (the counter retires in order); the
  // barrier publishes it to the group and frees the buffer read one stage earlier.
  const int trips = (p.steps - split * WK + stride - 1) / stride;
  for (int i = 0; i < trips; i += STG) {
#pragma unroll
    for (int s = 0; s < STG; ++s) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0((STG - 2) * TL::kLoads));
      if constexpr (WT > 1) __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      issue(k + (STG - 1) * stride, (s + STG - 1) % STG);
      __builtin_amdgcn_sched_barrier(0);
      mul(s);
      k += stride;
    }
  }
  __builtin_amdgcn_s_waitcnt(0);  // the trailing loads (zeros) have landed
  // lane l of a tile: token l % R, experts 8 (i / 4) + 4 (l / 32) + i % 4 (32x32) or 4 (l / 16) + i (16x16)
  float* out = p.out + (size_t)split * p.T * p.E;
  constexpr int Q = k32 ? 4 : 1;  // runs of 4 experts per lane
  auto store = [&](int m, int n, int q, f32x4 v) {
    const int t = t0 + m0 + m * R + r, e = e0 + n0 + n * R + 8 * q + 4 * g;
    if (t >= p.T) return;
    float* at = out + (size_t)t * p.E + e;
    if constexpr (W32) {
      if (splits == 1)  // (else the sum's launch looks)
        for (int j = 0; j < 4; ++j)
          if (v[j] != v[j] && e + j < p.E) v[j] = plain_dot(p, t, e + j);
    }
    if (e + 3 < p.E && (p.E & 3) == 0) {
      *(f32x4*)at = v;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e + j < p.E) at[j] = v[j];
    }
  };
  if constexpr (WK == 1) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < Q; ++q)
          store(m, n, q, f32x4{acc[m][n][4 * q], acc[m][n][4 * q + 1], acc[m][n][4 * q + 2], acc[m][n][4 * q + 3]});
  } else {
    static_assert(WK * BM * BN * 4 <= TL::kLds, "the sums fit the stages' space");
    __syncthreads();
    f32x4* red = (f32x4*)lds;  // [WK][WT][MT][NT][Q][64]
    constexpr int kRuns = MT * NT * Q;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < Q; ++q)
          red[(wave * kRuns + (m * NT + n) * Q + q) * 64 + lane] =
              f32x4{acc[m][n][4 * q], acc[m][n][4 * q + 1], acc[m][n][4 * q + 2], acc[m][n][4 * q + 3]};
    __syncthreads();
    // each group finishes its share of the runs
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      if (i % WK != kg) continue;
      f32x4 v = red[(wt * kRuns + i) * 64 + lane];
#pragma unroll
      for (int w = 1; w < WK; ++w) v += red[((w * WT + wt) * kRuns + i) * 64 + lane];
      store(i / Q / NT, i / Q % NT, i % Q, v);
    }
  }
}

// logits = the splits' partial sums, added in order (fp32 weights; bf16 ones never split)
__global__ __launch_bounds__(256) void router_sum_kernel(RouterParams p, float* __restrict__ out) {
  const size_t n = (size_t)p.T * p.E, i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float s = p.out[i];
  for (int k = 1; k < p.splits; ++k) s += p.out[(size_t)k * n + i];
  if (s != s) s = plain_dot(p, (int)(i / p.E), (int)(i % p.E));
  out[i] = s;
}

struct RouterPlan {
  int bm, bn;  // tile; bm 0: dot products
  int splits;
};
// The tile with the least rounds of 256 workgroups times what a round takes.  A small tile has the most
// bytes per flop and the shortest way through K; a taller one splits fp32 weights less often.  A round's
// time at H 7168, from runs at E 256, us (bf16, then fp32 weights):
//   16 x 16: T 256 7.7, 13; 32 x 32: T 1024 12.7, T 2048 24.0; 25.1, 46.6
//   32 x 64: T 2048 18.5, T 4096 35.0; 64 x 32: T 2048 33.4, T 4096 62.4
//   64 x 64: T 4096 23.8, T 8192 65 (its rounds slow down as more of x streams), T 16384 134
//   64 x 128: T 4096 39.5, T 8192 51, T 16384 105; 128 x 64: T 4096 92.8, T 8192 107, T 16384 214
//   128 x 128: T 8192 71, T 16384 79; 177, 181
// Splitting K costs a second launch of about 5 us.  It pays for fp32 weights between 64 x 32 and a full
// round of 128 x 64 tiles (T 4096: 55.4 in 2 splits, 62.4 with 64 x 32), never for bf16 ones (T 2048:
// 64 x 128 in 4 splits 18.2; T 4096 in 2: 26.9).  T 1 to 4: dot products 2.6 to 3.2, 16 x 16 5.8.
RouterPlan router_plan(int T, int H, int E, bool w_f32) {
  if (T <= 4) return RouterPlan{0, 1, 1};
  constexpr struct { int bm, bn; float us; } kTiles[2][6] = {
      {{16, 16, 8}, {32, 32, 13}, {32, 64, 18}, {64, 64, 26}, {64, 128, 51}, {128, 128, 78}},
      {{16, 16, 13}, {32, 32, 24}, {64, 32, 34}, {128, 64, 100}, {128, 128, 177}, {}}};
  RouterPlan best{};
  float least = INFINITY;
  for (const auto& t : kTiles[w_f32]) {
    if (t.bm == 0) break;
    const long long n = (long long)((T + t.bm - 1) / t.bm) * ((E + t.bn - 1) / t.bn);
    for (int splits = 1; splits == 1 || (w_f32 && t.bm == 128 && t.bn == 64 && splits <= 3 && n * splits <= 256); ++splits) {
      const float rounds = (float)((n * splits + 255) / 256);
      const float us = rounds * t.us * (float)H / (7168.0f * (float)splits) + (splits > 1 ? 5.0f : 0.0f);
      if (us < least) least = us, best = RouterPlan{t.bm, t.bn, splits};
    }
  }
  return best;
}

}  // namespace

size_t router_workspace_bytes(int T, int H, int E) {
  // Enough for the partial sums of every plan of up to T tokens with fp32 weights (bf16 ones never
  // split): a split plan has more than one round of 64 x 32 tiles, and at most 3 splits and 256 workgroups.
  if (H < 1024 || (long long)((T + 63) / 64) * ((E + 31) / 32) <= 256) return 0;
  return (size_t)std::min(3LL * T, 256LL * 128 / ((E + 63) / 64)) * E * 4;
}

hipError_t launch_router_logits(const RouterArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  const RouterPlan r = router_plan(a.T, a.H, a.E, a.w_f32);
  RouterParams p{(const uint8_t*)a.x, (const uint8_t*)a.w, r.splits > 1 ? a.partial : a.logits, a.T, a.H, a.E, 0,
                 (a.H + 63) / 64, r.splits};
  if (r.bm == 0) {
    auto go = [&](auto tt) {
      constexpr int TT = decltype(tt)::value;
      const dim3 grid((unsigned)a.E);
      if (a.w_f32) hipLaunchKernelGGL((router_dot_kernel<TT, true>), grid, dim3(256), 0, s, p);
      else hipLaunchKernelGGL((router_dot_kernel<TT, false>), grid, dim3(256), 0, s, p);
    };
    if (a.T == 1) go(std::integral_constant<int, 1>{});
    else if (a.T == 2) go(std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 4>{});
    return hipGetLastError();
  }
  p.n_tiles = (a.E + r.bn - 1) / r.bn;
  const unsigned m_tiles = (unsigned)((a.T + r.bm - 1) / r.bm);
  const dim3 grid = r.bm == 16 ? dim3((unsigned)p.n_tiles, m_tiles) : dim3(m_tiles * p.n_tiles * r.splits);
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(256), 0, s, p); };
  if (a.w_f32) {
    if (r.bm == 16) go(router_tile_kernel<16, 16, 1, 4, 4, true>);
    else if (r.bm == 32) go(router_tile_kernel<32, 32, 1, 4, 3, true>);
    else if (r.bm == 64) go(router_tile_kernel<64, 32, 1, 4, 2, true>);
    else if (r.bn == 64) go(router_tile_kernel<128, 64, 2, 2, 2, true>);
    else go(router_tile_kernel<128, 128, 4, 1, 3, true>);
  } else {
    if (r.bm == 16) go(router_tile_kernel<16, 16, 1, 4, 4, false>);
    else if (r.bm == 32 && r.bn == 32) go(router_tile_kernel<32, 32, 1, 4, 4, false>);
    else if (r.bm == 32) go(router_tile_kernel<32, 64, 1, 4, 3, false>);
    else if (r.bm == 64 && r.bn == 64) go(router_tile_kernel<64, 64, 1, 4, 2, false>);
    else if (r.bm == 64) go(router_tile_kernel<64, 128, 4, 1, 4, false>);
    else go(router_tile_kernel<128, 128, 4, 1, 4, false>);
  }
  if (r.splits > 1) {
    const dim3 sum_grid((unsigned)(((size_t)a.T * a.E + 255) / 256));
    hipLaunchKernelGGL(router_sum_kernel, sum_grid, dim3(256), 0, s, p, a.logits);
  }
  return hipGetLastError();
}

}  // namespace moe
