// Top-k of one token's router logits by one wavefront, and the wavefront
// reductions it uses: shared by the top-k kernel and the few-token layer, which
// routes inside its first launch.  Internal to the library.
#pragma once
#include "device.h"

namespace moe {

// Order-preserving map of a float key to 32 bits (larger key, larger value;
// -0 and +0 equal, as the float comparison has them).
MOE_DEV uint32_t key_bits(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The wave's largest 64-bit (key, ~index) word, uniform: butterflies inside each
// row of 16 lanes by DPP (quad swaps, half-row and row mirrors), then the four
// row results read into scalars.  (Cross-lane shuffles through the LDS crossbar
// made each of the k selection rounds a chain of 18 round trips.)
template <int CTRL>
MOE_DEV uint64_t dpp_max_u64(uint64_t x) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)x, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(x >> 32), CTRL, 0xF, 0xF, false);
  const uint64_t y = ((uint64_t)hi << 32) | lo;
  return y > x ? y : x;
}
MOE_DEV uint64_t wave_max_u64(uint64_t x) {
  x = dpp_max_u64<0xB1>(x);   // quad_perm [1,0,3,2]
  x = dpp_max_u64<0x4E>(x);   // quad_perm [2,3,0,1]
  x = dpp_max_u64<0x141>(x);  // row_half_mirror
  x = dpp_max_u64<0x140>(x);  // row_mirror
  uint64_t m = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint64_t v = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), 16 * r) << 32) |
                       (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, 16 * r);
    m = v > m ? v : m;
  }
  return m;
}

// The wave's maximum and sum of a float (uniform), by the same DPP butterflies
// and row read-outs; the sum adds the four row sums in row order.
template <int CTRL>
MOE_DEV float dpp_f32(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}
MOE_DEV float wave_max_f32(float x) {
  x = fmaxf(x, dpp_f32<0xB1>(x));
  x = fmaxf(x, dpp_f32<0x4E>(x));
  x = fmaxf(x, dpp_f32<0x141>(x));
  x = fmaxf(x, dpp_f32<0x140>(x));
  float m = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 0));
#pragma unroll
  for (int r = 1; r < 4; ++r)
    m = fmaxf(m, __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 16 * r)));
  return m;
}
MOE_DEV float wave_sum_f32(float x) {
  x += dpp_f32<0xB1>(x);
  x += dpp_f32<0x4E>(x);
  x += dpp_f32<0x141>(x);
  x += dpp_f32<0x140>(x);
  float m = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 0));
#pragma unroll
  for (int r = 1; r < 4; ++r) m += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 16 * r));
  return m;
}

// The wave's sum of a double, the same way.
template <int CTRL>
MOE_DEV double dpp_f64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
MOE_DEV double wave_sum_f64(double x) {
  x += dpp_f64<0xB1>(x);
  x += dpp_f64<0x4E>(x);
  x += dpp_f64<0x141>(x);
  x += dpp_f64<0x140>(x);
  double m = 0.0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint64_t v = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 16 * r) << 32 |
                       (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 16 * r);
    m += __builtin_bit_cast(double, v);
  }
  return m;
}

// The larger of a lane's value and a DPP neighbour's.
template <int CTRL>
MOE_DEV uint32_t dpp_max_u32(uint32_t x) {
  const uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xF, 0xF, false);
  return y > x ? y : x;
}

// One token's routing by one wavefront.  Each lane holds logits e = lane + 64*i
// (i < 8, so E <= 512), k rounds of wave-wide argmax with key (logit + bias desc, index asc), then a
// softmax over the k selected logits.  The optional per-expert bias (the
// routing_bias of bias-aware methods on the MoEActivationPack page) only ranks
// the experts: the weights come from the logits themselves.  Lane s < k returns
// slot s's expert and weight.
template <bool FAST>
MOE_DEV void route_token_topk(const float* __restrict__ row, const float* __restrict__ bias, int E, int k, int& my_i,
                              float& my_w) {
  const int lane = lane_id();
  float v[8], key[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    int e = lane + 64 * i;
    float x = e < E ? row[e] : -INFINITY;
    v[i] = (x != x) ? -INFINITY : x;  // NaN ranks as -inf
    const float kb = (bias != nullptr && e < E) ? v[i] + bias[e] : v[i];
    key[i] = (kb != kb) ? -INFINITY : kb;
  }
  unsigned taken = 0;
  float my_v = -INFINITY;
  my_i = 0;
  for (int s = 0; s < k; ++s) {
    float bk = -INFINITY, bv = -INFINITY;
    int bi = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int e = lane + 64 * i;
      bool ok = e < E && !((taken >> i) & 1u);
      if (ok && (key[i] > bk || (key[i] == bk && e < bi))) {
        bk = key[i];
        bv = v[i];
        bi = e;
      }
    }
    // the wave's winner: largest key, then smallest index (a lane without a
    // candidate, ~0x7FFFFFFF, loses to any expert at an equal key)
    const uint64_t w = wave_max_u64(((uint64_t)key_bits(bk) << 32) | (uint32_t)~bi);
    bi = (int)~(uint32_t)w;
    bv = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, bv), bi & 63));
    if ((bi & 63) == lane) taken |= 1u << (bi >> 6);
    if (lane == s) {
      my_v = bv;
      my_i = bi;
    }
  }
  // the largest selected logit (the first one when there is no bias)
  const float vmax = wave_max_f32(lane < k ? my_v : -INFINITY);
  float ex = 0.0f;
  if (lane < k) ex = FAST ? __builtin_amdgcn_exp2f((my_v - vmax) * 1.4426950408889634f) : expf(my_v - vmax);
  const float sum = wave_sum_f32(ex);
  my_w = FAST ? ex * __builtin_amdgcn_rcpf(sum) : ex / sum;
}

}  // namespace moe
