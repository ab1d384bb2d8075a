// Router logits: logits[t, e] = sum over h of x[t, h] * W[e, h], x bf16 and W bf16
// or fp32, fp32 sums: what FromLogits routing (the routing_input_mode entry of the
// MoEActivationPack page) starts from.
//
// v_mfma_f32_16x16x32_bf16 with the router's rows as the first operand and the
// tokens as the second.  fp32 weights are split into three bf16 terms whose sum
// holds all 24 bits of the weight (w = w0 + w1 + w2 exactly, barring underflow),
// each multiplied on the matrix cores: bf16 products are exact in fp32, so the
// result has the error of an fp32 sum.
#include "gemm_common.h"
#include "layer.h"

namespace moe {

namespace {

constexpr int kRouterWaves = 8;

struct RouterParams {
  const uint8_t* x;
  const uint8_t* w;
  float* out;  // logits, or the partial sums [splits][T][E]
  int T, H, E;
  int n_tiles;   // expert tiles
  int steps;     // K-steps of 64
  int splits;    // workgroups that share a tile's K-steps
};

// Three bf16 terms of 8 fp32 values: each is the rounding of what the ones before leave.
MOE_DEV void split3(const f32x4 a, const f32x4 b, i32x4 (&o)[3]) {
  float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
  for (int s = 0; s < 3; ++s)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t r = bf16x2_rne(v[2 * q], v[2 * q + 1]);
      o[s][q] = (int)r;
      const float lo = __uint_as_float(r << 16), hi = __uint_as_float(r & 0xFFFF0000u);
      // an infinite or NaN weight is its first term alone
      v[2 * q] = s > 0 || fabsf(lo) < INFINITY ? v[2 * q] - lo : 0.0f;
      v[2 * q + 1] = s > 0 || fabsf(hi) < INFINITY ? v[2 * q + 1] - hi : 0.0f;
    }
}

// A workgroup computes 16 MT tokens x 16 NT experts; its waves (and the workgroups
// of a split) take every kRouterWaves-th K-step of 64, and their sums are added
// in wave order.
template <int MT, int NT, bool W32>
__global__ __launch_bounds__(64 * kRouterWaves) void router_mfma_kernel(RouterParams p) {
  constexpr int kFrag = W32 ? 2 : 1;  // 16-byte pieces of 8 weights
  __shared__ f32x4 red[kRouterWaves][MT * NT][64];
  const int tid = threadIdx.x, lane = lane_id(), g = lane >> 4, r16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int split = blockIdx.x % p.splits, tile = blockIdx.x / p.splits;
  const int t0 = tile / p.n_tiles * (16 * MT), e0 = tile % p.n_tiles * (16 * NT);
  const uint32_t xrow = (uint32_t)p.H * 2, wrow = (uint32_t)p.H * (W32 ? 4 : 2);
  const __amdgpu_buffer_rsrc_t x_rs = make_rsrc(p.x + (size_t)t0 * xrow, (uint32_t)min(16 * MT, p.T - t0) * xrow);
  const __amdgpu_buffer_rsrc_t w_rs = make_rsrc(p.w + (size_t)e0 * wrow, (uint32_t)min(16 * NT, p.E - e0) * wrow);
  uint32_t xo[MT], wo[NT];  // rows past the last one lie past the resource: zeros
#pragma unroll
  for (int m = 0; m < MT; ++m) xo[m] = (uint32_t)(16 * m + r16) * xrow + 16u * g;
#pragma unroll
  for (int n = 0; n < NT; ++n) wo[n] = (uint32_t)(16 * n + r16) * wrow + 16u * kFrag * g;
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Stage {
    i32x4 x[MT][2], w[NT][2][kFrag];
  };
  auto load = [&](Stage& s, int k) {
    const uint32_t dead = oob_if(k >= p.steps);
    // H is a multiple of 32: the last K-step may hold 32 elements
    const uint32_t dead2 = oob_if(k * 64 + 32 >= p.H) | dead;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      s.x[m][0] = bload16(x_rs, xo[m] | dead, (uint32_t)k * 128u);
      s.x[m][1] = bload16(x_rs, (xo[m] + 64u) | dead2, (uint32_t)k * 128u);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int f = 0; f < kFrag; ++f) {
        s.w[n][0][f] = bload16(w_rs, (wo[n] + 16u * f) | dead, (uint32_t)k * 128u * kFrag);
        s.w[n][1][f] = bload16(w_rs, (wo[n] + 64u * kFrag + 16u * f) | dead2, (uint32_t)k * 128u * kFrag);
      }
  };
  auto mul = [&](const Stage& s) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        i32x4 wf[W32 ? 3 : 1];
        if constexpr (W32) {
          split3(__builtin_bit_cast(f32x4, s.w[n][hh][0]), __builtin_bit_cast(f32x4, s.w[n][hh][1]), wf);
        } else {
          wf[0] = s.w[n][hh][0];
        }
#pragma unroll
        for (int q = (W32 ? 2 : 0); q >= 0; --q)  // the smallest term first
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wf[q]),
                                                                __builtin_bit_cast(bf16x8, s.x[m][hh]), acc[m][n], 0, 0, 0);
      }
  };
  const int stride = kRouterWaves * p.splits;
  int k = split * kRouterWaves + wave;
  Stage a, b;
  load(a, k);
  while (k < p.steps) {
    load(b, k + stride);
    mul(a);
    load(a, k + 2 * stride);
    mul(b);
    k += 2 * stride;
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) red[wave][m * NT + n][lane] = acc[m][n];
  __syncthreads();
  // lane l of tile (m, n): token 16 m + l % 16, experts 16 n + 4 (l / 16) ...
  float* out = p.out + (size_t)split * p.T * p.E;
  for (int i = tid; i < MT * NT * 64; i += 64 * kRouterWaves) {
    const int mn = i >> 6, l = i & 63;
    f32x4 s = red[0][mn][l];
#pragma unroll
    for (int w = 1; w < kRouterWaves; ++w) s += red[w][mn][l];
    const int t = t0 + mn / NT * 16 + (l & 15), e = e0 + mn % NT * 16 + 4 * (l >> 4);
    if (t >= p.T) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (e + q < p.E) out[(size_t)t * p.E + e + q] = s[q];
  }
}

// logits = the splits' partial sums, added in order
__global__ __launch_bounds__(256) void router_sum_kernel(const float* __restrict__ part, float* __restrict__ out,
                                                         size_t n, int splits) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float s = part[i];
  for (int k = 1; k < splits; ++k) s += part[(size_t)k * n + i];
  out[i] = s;
}

struct RouterPlan {
  int tile;  // tokens and experts of a tile: 16, 32 or 64
  int splits;
};
RouterPlan router_plan(int, int, int) { return RouterPlan{16, 1}; }

}  // namespace

size_t router_workspace_bytes(int T, int H, int E) {
  const RouterPlan r = router_plan(T, H, E);
  return r.splits > 1 ? (size_t)r.splits * T * E * 4 : 0;
}

hipError_t launch_router_logits(const RouterArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  const RouterPlan r = router_plan(a.T, a.H, a.E);
  const int m_tiles = (a.T + r.tile - 1) / r.tile, n_tiles = (a.E + r.tile - 1) / r.tile;
  RouterParams p{(const uint8_t*)a.x, (const uint8_t*)a.w, r.splits > 1 ? a.partial : a.logits, a.T, a.H, a.E, n_tiles,
                 (a.H + 63) / 64, r.splits};
  const dim3 grid((unsigned)(m_tiles * n_tiles * r.splits)), block(64 * kRouterWaves);
  if (a.w_f32) hipLaunchKernelGGL((router_mfma_kernel<1, 1, true>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((router_mfma_kernel<1, 1, false>), grid, block, 0, s, p);
  if (r.splits > 1) {
    const size_t n = (size_t)a.T * a.E;
    hipLaunchKernelGGL(router_sum_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a.partial, a.logits, n,
                       r.splits);
  }
  return hipGetLastError();
}

}  // namespace moe
