// Internal launchers of the products by expert outside the fused layer (bf16 with their
// gradients, MXFP4), of the SwiGLU between them and of the MXFP4 quantiser.  Not part of the
// public C ABI.
#pragma once
#include "launch.h"

namespace moe {

// What a plan row stands for in a tensor: the row itself, token src_info / k, or pair src_info.
enum class Rows : int { PLAN = 0, TOKEN = 1, PAIR = 2 };

struct GroupedArgs {
  int E, topk, T;
  const int* start;     // expert_start_indices [E+1]
  const int* src_info;  // [T*k]
  int n, k;             // out columns, summed length (wgrad: dout's and a's columns)
  const void* a;        // rows of k bf16, or of k / 2 bytes of E2M1
  const void* a_sf;     // MXFP4: [.., k/32]
  Rows a_rows;
  const void* w;        // [E, n, k] ([E, k, n] with w_kn)
  const void* w_sf;     // MXFP4: [E, n, k/32]
  bool w_kn;
  void* out;            // rows of n, bf16 or fp32
  bool out_f32;
  Rows out_rows;
};
// whether a launch's grid holds the tiles of the smallest shape
bool grouped_gemm_fits(int npairs, int E, int n);
bool grouped_wgrad_fits(int E, int n, int k);
hipError_t launch_grouped_gemm(const GroupedArgs& a, hipStream_t s);
hipError_t launch_grouped_gemm_mxfp4(const GroupedArgs& a, hipStream_t s);

struct WgradArgs {
  int E, topk, T;
  const int* start;
  const int* src_info;
  int n, k;
  const void* dout;  // rows of n bf16
  Rows dout_rows;
  const void* a;     // rows of k bf16
  Rows a_rows;
  void* dw;          // [E, n, k] bf16 or fp32
  bool dw_f32, accumulate;
};
hipError_t launch_grouped_wgrad(const WgradArgs& a, hipStream_t s);

// rows of `cols` bf16 or fp32, `stride` elements apart, to MXFP4 (and, values != nullptr, to what the codes stand for)
hipError_t launch_quantize_mxfp4(const void* x, bool x_f32, long long rows, int cols, long long stride, void* q,
                                 void* sf, void* values, hipStream_t s);

struct SwigluArgs {
  int E, npairs, I;
  const int* start;   // rows start[E] and beyond are left as they are
  float clamp;
  bool fast;
  const void* gu;     // [rows, 2I] bf16: gate, up
  const void* dh;     // [rows, I] bf16, or nullptr: forward
  void* h;            // [rows, I] bf16 or nullptr
  void* q;            // MXFP4 of the unrounded h, or nullptr
  void* sf;
  void* dgu;          // [rows, 2I] bf16 (backward)
};
hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s);

}  // namespace moe
