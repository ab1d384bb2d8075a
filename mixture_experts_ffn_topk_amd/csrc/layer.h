// Internal launchers of the operators around the expert FFN (the norm ahead of
// it and the router's logits) and of the routed layer for few tokens.  Not part
// of the public C ABI.
#pragma once
#include "launch.h"

namespace moe {

// ---------------------------------------------------------------- residual + RMS norm
// The widest row the norm kernel holds in registers.
constexpr int kNormMaxHidden = 32768;
struct NormArgs {
  Fmt fmt;  // BF16 / NV4: bf16 activations (x_q, x_sf unused)
  int T, H;
  const void* x;         // [T, H] bf16 or fp32
  const void* residual;  // [T, H] bf16 or fp32, or nullptr
  const void* weight;    // [H] bf16 or fp32
  bool x_f32, residual_f32, weight_f32;
  float eps, x_gs;       // x_gs: NVFP4's global scale of the activations
  void* residual_out;    // [T, H], residual's type
  void* x_norm;          // [T, H] bf16 or nullptr
  void* x_q;             // the format's activations or nullptr
  void* x_sf;
};
hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s);

// ---------------------------------------------------------------- router logits
struct RouterArgs {
  int T, H, E;
  const void* x;  // [T, H] bf16
  const void* w;  // [E, H] bf16 or fp32
  bool w_f32;
  float* logits;  // [T, E]
  float* partial; // router_workspace_bytes(T, H, E)
};
size_t router_workspace_bytes(int T, int H, int E);  // never shrinks with T
hipError_t launch_router_logits(const RouterArgs& a, hipStream_t s);

// ---------------------------------------------------------------- the layer for few tokens
constexpr int kFewMaxTokens = 32;
struct FewArgs {
  Fmt fmt;
  int T, E, topk, H, I;
  float clamp;
  bool fast;
  const void* ids;       // [T, k]: the routing, also where the first launch writes it (logits != nullptr)
  bool ids64;
  const float* topk_w;   // [T, k]
  const float* logits;   // [T, E] or nullptr: the first launch routes
  const float* bias;     // [E] or nullptr
  const void* x;
  const void* x_sf;
  const void* w13;  // prepared layout
  const void* w13_sf;
  const void* w2;
  const void* w2_sf;
  const float* w13_gs;
  const float* w2_gs;
  const float* c_scales;
  void* h;        // the buffers of few_buffers
  void* h_sf;
  void* tables;
  void* arrived;
  void* part;
  const void* shared;
  const void* residual;
  void* out;
  bool out_f32;
};
// Whether the first launch can route from logits itself (else the top-k launch
// comes before it).
bool few_routes_in_launch(int T);
struct FewBuffers {
  size_t h, h_sf, tables, arrived, part;  // bytes
};
FewBuffers few_buffers(Fmt f, int T, int topk, int E, int H, int I);
hipError_t launch_few(const FewArgs& a, hipStream_t s);

}  // namespace moe
