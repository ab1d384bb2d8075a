// Products by expert on a routing plan's rows, outside the fused layer:
//
//   forward    out[o(r), j]  = sum over i of a[s(r), i] * w[e][j][i]        (bf16, or MXFP4 x MXFP4)
//   gradient   out[o(r), j]  = sum over i of a[s(r), i] * w[e][i][j]        (w_kn)
//   weights    dw[e][j][i]  (+)= sum over e's rows r of dout[s(r), j] * a[s'(r), i]
//
// for the rows r of expert e, start[e] <= r < start[e+1].  Weights are canonical (they change with every training step,
// so nothing is laid out ahead).
//
// Both operands go through LDS by direct-to-LDS loads of whole lines.  P is the operand whose rows become the output's
// contiguous columns (the weights; a for the weight gradient), Q the one whose rows become its rows; P is the first MFMA
// operand, so that a lane ends with 4 consecutive columns of a row.  An operand whose summed index is its contiguous one
// is staged as rows of 128 bytes and read with ds_read_b128; the others (T: transposed) as 64 summed rows of all the
// tile's columns, read with ds_read_b64_tr_b16, which hands a lane 4 summed rows of its column.
#include <algorithm>

#include "gemm_common.h"
#include "grouped.h"

namespace moe {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

enum class Op { FWD, GRAD, WGRAD, MX };

// Where plan row r, pair src = src_info[r], lies in a tensor: at r, src or src / k.  (A quotient by a product is exact for
// src below 2^27, and there are at most 2^26 pairs: the error of ceil(2^32 / k) is below k <= 32.)
struct Place {
  uint32_t inverse;  // ceil(2^32 / k); 0: the pair itself
  int whole;         // -1: the pair itself, else 0
  int gathered;      // -1: by src, 0: r
  int places;        // the tensor's rows: a plan that is none reads nothing past them
  MOE_DEV int of(int r, int src) const {
    const int at = min(max((int)__umulhi((uint32_t)src, inverse) + (src & whole), 0), places - 1);
    return (at & gathered) | (r & ~gathered);
  }
};

struct GroupedParams {
  const int* start;
  const int* src_info;
  int E, npairs;
  const uint8_t* P;      // weights, or a (WGRAD)
  const uint8_t* Q;      // a's rows, or dout's (WGRAD)
  const uint8_t* P_sf;   // MXFP4 scales
  const uint8_t* Q_sf;
  long long p_expert;    // bytes of one expert's weights
  long long p_sf_expert;
  long long p_ld, q_ld;  // bytes between rows as they lie in memory
  int p_cols, q_cols;    // extents of the output (q_cols: WGRAD only, else the expert's rows)
  int K;                 // summed length (WGRAD: the expert's rows)
  int sf_row;            // MXFP4: K / 32
  Place q_place, p_place;
  void* out;
  long long out_ld;      // elements
  long long out_expert;  // WGRAD: elements of one expert's dw
  int out_pair;          // rows go to src_info[r]
  int accumulate;
  int p_tiles, q_tiles;  // q_tiles: WGRAD; else the worst case over all experts
};

// 16 bytes that masked lanes load.
__device__ __attribute__((aligned(16))) const uint32_t zero16[4] = {0, 0, 0, 0};

MOE_DEV void lds_copy16(const void* g, void* l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g, (LDS3 void*)l, 16, 0, 0);
}

MOE_DEV int wave_scan(int v) {  // inclusive
  const int lane = lane_id();
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  return v;
}

struct TileAt {
  int expert, lo, hi;  // the expert's rows
  int q, p;            // tile indices within the expert
};

// start[e], made safe against a plan that is none.
MOE_DEV int row_at(const GroupedParams& p, int e) { return min(max(p.start[e], 0), p.npairs); }

// The tile of this workgroup; false: there is none.  Tiles lie expert by expert, in groups of GQ q-tiles, within a group
// p-tile by p-tile: the workgroups that an XCD runs at once then share few operand panels in its L2.
template <bool WGRAD, int BQ, int GQ>
MOE_DEV bool find_tile(const GroupedParams& p, TileAt* t) {
  const int lane = lane_id();
  int L, within = 0;
  if (WGRAD) {
    const int per = p.q_tiles * p.p_tiles;
    L = xcd_remap(blockIdx.x, gridDim.x);
    t->expert = L / per;
    within = L - t->expert * per;
    t->lo = row_at(p, t->expert);
    t->hi = max(t->lo, row_at(p, t->expert + 1));
  } else {
    int total = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const int e = e0 + lane;
      int c = 0;
      if (e < p.E) c = (max(0, row_at(p, e + 1) - row_at(p, e)) + BQ - 1) / BQ;
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) c += __shfl_xor(c, d);
      total += c;
    }
    const int G = min(total * p.p_tiles, (int)gridDim.x);
    if ((int)blockIdx.x >= G) return false;
    L = xcd_remap(blockIdx.x, G);
    int before = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const int e = e0 + lane;
      int lo = 0, hi = 0;
      if (e < p.E) lo = row_at(p, e), hi = max(lo, row_at(p, e + 1));
      const int mine = (hi - lo + BQ - 1) / BQ * p.p_tiles, upto = before + wave_scan(mine);
      const unsigned long long found = __ballot(upto > L);
      if (found) {
        const int at = __ffsll(found) - 1;
        t->expert = e0 + at;
        t->lo = __shfl(lo, at);
        t->hi = __shfl(hi, at);
        within = L - __shfl(upto - mine, at);
        break;
      }
      before = __shfl(upto, 63);
    }
  }
  t->expert = __builtin_amdgcn_readfirstlane(t->expert);
  t->lo = __builtin_amdgcn_readfirstlane(t->lo);
  t->hi = __builtin_amdgcn_readfirstlane(t->hi);
  within = __builtin_amdgcn_readfirstlane(within);
  const int qt = WGRAD ? p.q_tiles : (t->hi - t->lo + BQ - 1) / BQ;
  const int group = within / (GQ * p.p_tiles), q0 = group * GQ, size = min(GQ, qt - q0);
  const int in = within - group * GQ * p.p_tiles;
  t->p = in / size;
  t->q = q0 + in - t->p * size;
  return true;
}

// Where 16-byte chunk c of row r lies among its row's eight (rows of 128 bytes): a 32-row operand's lanes r and r + 16
// are read together, so both row bits take part.
MOE_DEV int swz(int r) { return (r & 7) ^ ((r >> 4) & 1); }

// Transposed operands: the 32-byte unit u of summed row r lies at u ^ trx(r), so that the 4 rows x 2 units that 32 lanes
// read lie in different banks.
template <int B>
MOE_DEV int trx(int r) {
  return B >= 256 ? (2 * (r & 3)) | (r & 8) : 2 * (r & 3);
}

// ---------------------------------------------------------------- tiles
// BP x BQ outputs per workgroup, WP x WQ waves, each TP x TQ MFMA tiles of 32 x 32.
template <Op O, int BP, int BQ, int WP, int WQ>
struct GTile {
  static constexpr int kWaves = WP * WQ, kThreads = 64 * kWaves;
  static constexpr int TP = BP / 32 / WP, TQ = BQ / 32 / WQ;
  static constexpr bool kTP = O == Op::GRAD || O == Op::WGRAD, kTQ = O == Op::WGRAD;
  static constexpr int kPBytes = BP * 128, kQBytes = BQ * 128, kStage = kPBytes + kQBytes;
  static constexpr int kSf = O == Op::MX ? (BP + BQ) * 8 : 0;  // a K-step's scales: 8 bytes a row
  static constexpr int kLp = kPBytes / (16 * kThreads), kLq = kQBytes / (16 * kThreads);  // loads per lane and stage
  static constexpr int kStages = 2 * kStage + 2 * kSf;
  // the output on its way to memory: rows of BP fp32 or bf16, as many at once as fit
  static constexpr int kLds = kStages;
  static constexpr int kBK = O == Op::MX ? 256 : 64;  // elements of a K-step
};

template <Op O, int BP, int BQ, int WP, int WQ, bool F32, int GQ>
__global__ __launch_bounds__(64 * WP * WQ, 2) void grouped_kernel(GroupedParams p) {
  using TL = GTile<O, BP, BQ, WP, WQ>;
  constexpr bool MX = O == Op::MX, WG = O == Op::WGRAD, kTP = TL::kTP, kTQ = TL::kTQ;
  constexpr int TP = TL::TP, TQ = TL::TQ, BK = TL::kBK, kThreads = TL::kThreads;
  __shared__ __attribute__((aligned(16))) uint8_t lds[TL::kLds];
  TileAt t;
  if (!find_tile<WG, BQ, GQ>(p, &t)) return;
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wave % WP, wq = wave / WP, h = lane >> 5, r32 = lane & 31;
  const int p0 = t.p * BP;
  const int rows = t.hi - t.lo;
  const int q0 = t.q * BQ;                        // of the expert's rows (WGRAD: of dout's columns)
  const int q_last = (WG ? p.q_cols : rows) - 1;  // the last row (column) of the output there is
  const int K = WG ? rows : p.K, steps = (K + BK - 1) / BK;
  const uint8_t* P = p.P + (long long)t.expert * p.p_expert;

  // ---------------------------------------------------------------- what each lane loads
  const uint8_t* pp[TL::kLp];
  const uint8_t* qq[TL::kLq];
  int p_chunk = 0, q_chunk = 0;  // 16-byte chunk of the row
  constexpr int kPC = BP / 8, kQC = BQ / 8;  // T operands: chunks per summed row
  if constexpr (!kTP) {
    p_chunk = (lane & 7) ^ swz((wave * 8 + (lane >> 3)));
#pragma unroll
    for (int i = 0; i < TL::kLp; ++i) {
      const int r = min(p0 + (i * TL::kWaves + wave) * 8 + (lane >> 3), p.p_cols - 1);
      pp[i] = P + r * p.p_ld + p_chunk * 16;
    }
  } else {
    const int kr = wave * (64 / kPC) + lane / kPC, slot = lane % kPC;
    p_chunk = (((slot >> 1) ^ trx<BP>(kr)) << 1) | (slot & 1);
    p_chunk = min(p0 / 8 + p_chunk, p.p_cols / 8 - 1);
#pragma unroll
    for (int i = 0; i < TL::kLp; ++i)
      pp[i] = P + (long long)(i * TL::kWaves * (64 / kPC) + kr) * p.p_ld + p_chunk * 16;
  }
  if constexpr (!kTQ) {
    q_chunk = (lane & 7) ^ swz((wave * 8 + (lane >> 3)));
#pragma unroll
    for (int i = 0; i < TL::kLq; ++i) {
      long long r = t.lo + min(q0 + (i * TL::kWaves + wave) * 8 + (lane >> 3), q_last);
      if (p.q_place.gathered) r = p.q_place.of(0, p.src_info[r]);
      qq[i] = p.Q + r * p.q_ld + q_chunk * 16;
    }
  } else {
    const int kr = wave * (64 / kQC) + lane / kQC, slot = lane % kQC;
    q_chunk = (((slot >> 1) ^ trx<BQ>(kr)) << 1) | (slot & 1);
    q_chunk = min(q0 / 8 + q_chunk, p.q_cols / 8 - 1);
  }
  // WGRAD: src_info of the summed rows, one K-step ahead of their loads (read also where the rows are the plan's own: a
  // test would split the loop into blocks)
  int p_src[WG ? TL::kLp : 1], q_src[WG ? TL::kLq : 1];
  const int p_kr = wave * (64 / kPC) + lane / kPC, q_kr = wave * (64 / kQC) + lane / kQC;
  auto places = [&](int ks) {
    if constexpr (WG) {
#pragma unroll
      for (int i = 0; i < TL::kLp; ++i)
        p_src[i] = p.src_info[min(t.lo + ks * BK + i * TL::kWaves * (64 / kPC) + p_kr, t.hi - 1)];
#pragma unroll
      for (int i = 0; i < TL::kLq; ++i)
        q_src[i] = p.src_info[min(t.lo + ks * BK + i * TL::kWaves * (64 / kQC) + q_kr, t.hi - 1)];
    }
  };
  // MXFP4: thread -> a row's scales of a K-step, 8 bytes from an address that may be odd
  typedef const __attribute__((address_space(1))) uint32_t* GlobalWord;
  const uint8_t* sf_base = nullptr;
  uint32_t sf_shift = 0;
  uint32_t sf[3] = {0, 0, 0};
  static_assert(!MX || BP + BQ == kThreads, "one thread per row of scales");
  if constexpr (MX) {
    const bool isp = tid < BP;
    long long at;
    if (isp) {
      at = (long long)t.expert * p.p_sf_expert + (long long)min(p0 + tid, p.p_cols - 1) * p.sf_row;
    } else {
      long long r = t.lo + min(q0 + min(tid - BP, BQ - 1), q_last);
      if (p.q_place.gathered) r = p.q_place.of(0, p.src_info[r]);
      at = r * p.sf_row;
    }
    const uint8_t* s = (isp ? p.P_sf : p.Q_sf) + at;
    sf_shift = (uint32_t)((uintptr_t)s & 3);
    sf_base = s - sf_shift;
  }
  // the aligned words that hold a row's scales [8 ks, 8 ks + 8) (those past its end are not read)
  auto load_sf = [&](int ks) {
    if constexpr (MX) {
      const int left = (int)sf_shift + p.sf_row - 8 * ks;  // bytes from the first word to the row's end
      const GlobalWord w = (GlobalWord)(sf_base + 8 * ks), none = (GlobalWord)zero16;
#pragma unroll
      for (int i = 0; i < 3; ++i) sf[i] = *(4 * i < left ? w + i : none);
    }
  };
  auto store_sf = [&](int ks, int buf) {
    if constexpr (MX) {
      const int left = p.sf_row - 8 * ks;
      uint32_t lo = __builtin_amdgcn_alignbyte(sf[1], sf[0], sf_shift), hi = __builtin_amdgcn_alignbyte(sf[2], sf[1], sf_shift);
      // blocks past K: scale 2^-127 on codes of zero
      const uint64_t keep = left >= 8 ? ~0ull : left <= 0 ? 0ull : (1ull << (8 * left)) - 1;
      *(uint2*)(lds + 2 * TL::kStage + buf * TL::kSf + tid * 8) = uint2{lo & (uint32_t)keep, hi & (uint32_t)(keep >> 32)};
    }
  };

  auto issue = [&](int ks, int buf) {
    uint8_t* lp = lds + buf * TL::kStage + wave * 1024;
    uint8_t* lq = lp + TL::kPBytes;
    if constexpr (WG) {
#pragma unroll
      for (int i = 0; i < TL::kLp; ++i) {
        const int r = t.lo + ks * BK + i * TL::kWaves * (64 / kPC) + p_kr;
        const uint8_t* g = p.P + (long long)p.p_place.of(r, p_src[i]) * p.p_ld + p_chunk * 16;
        lds_copy16(r < t.hi ? g : (const uint8_t*)zero16, lp + i * TL::kWaves * 1024);
      }
#pragma unroll
      for (int i = 0; i < TL::kLq; ++i) {
        const int r = t.lo + ks * BK + i * TL::kWaves * (64 / kQC) + q_kr;
        const uint8_t* g = p.Q + (long long)p.q_place.of(r, q_src[i]) * p.q_ld + q_chunk * 16;
        lds_copy16(r < t.hi ? g : (const uint8_t*)zero16, lq + i * TL::kWaves * 1024);
      }
      return;
    }
    constexpr int kPer = MX ? 32 : 8;  // elements of a chunk
#pragma unroll
    for (int i = 0; i < TL::kLp; ++i) {
      const int at = kTP ? ks * BK + i * TL::kWaves * (64 / kPC) + p_kr : ks * BK + p_chunk * kPer;
      lds_copy16(at < K ? pp[i] : (const uint8_t*)zero16, lp + i * TL::kWaves * 1024);
      pp[i] += kTP ? 64 * p.p_ld : 128;
    }
#pragma unroll
    for (int i = 0; i < TL::kLq; ++i) {
      lds_copy16(ks * BK + q_chunk * kPer < K ? qq[i] : (const uint8_t*)zero16, lq + i * TL::kWaves * 1024);
      qq[i] += 128;
    }
  };

  // ---------------------------------------------------------------- fragments
  i32x4 fp[2][TP], fq[2][TQ];
  uint32_t sp[TP], sq[TQ];
  auto frag = [&](const uint8_t* base, bool tr, int ld, int tile, int s) -> i32x4 {
    if (!tr) {
      const int c = (MX ? 4 * h + s : 2 * s + h) ^ swz(r32);
      return *(const i32x4*)(base + (tile * 32 + r32) * 128 + c * 16);
    }
    const int row = 16 * s + 8 * h + ((lane & 15) >> 2), u = tile * 2 + ((lane >> 4) & 1);
    const uint8_t* a = base + row * ld + ((u ^ (ld >= 512 ? trx<256>(row) : trx<128>(row))) << 5) + (lane & 3) * 8;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS3 s16x4*)a);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS3 s16x4*)(a + 4 * ld));
    return __builtin_bit_cast(i32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto read = [&](int buf, int s, int set) {
    const uint8_t* b = lds + buf * TL::kStage;
#pragma unroll
    for (int i = 0; i < TP; ++i) fp[set][i] = frag(b, kTP, BP * 2, wp * TP + i, s);
#pragma unroll
    for (int i = 0; i < TQ; ++i) fq[set][i] = frag(b + TL::kPBytes, kTQ, BQ * 2, wq * TQ + i, s);
  };
  // a K-step's scales: byte s of a lane's word belongs to sub-step s
  auto read_sf = [&](int buf) {
    if constexpr (MX) {
      const uint32_t* f = (const uint32_t*)(lds + 2 * TL::kStage + buf * TL::kSf);
#pragma unroll
      for (int i = 0; i < TP; ++i) sp[i] = f[((wp * TP + i) * 32 + r32) * 2 + h];
#pragma unroll
      for (int i = 0; i < TQ; ++i) sq[i] = f[(BP + (wq * TQ + i) * 32 + r32) * 2 + h];
    }
  };
  f32x16 acc[TP][TQ];
#pragma unroll
  for (int i = 0; i < TP; ++i)
#pragma unroll
    for (int j = 0; j < TQ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  auto mma = [&](auto sub, int set) {
    constexpr int S = decltype(sub)::value;
#pragma unroll
    for (int j = 0; j < TQ; ++j)
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        if constexpr (MX) {
          const i32x4 a = fp[set][i], b = fq[set][j];
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0}, i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, acc[i][j], 4, 4, S,
              (int)sp[i], S, (int)sq[j]);
        } else {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, fp[set][i]),
                                                              __builtin_bit_cast(bf16x8, fq[set][j]), acc[i][j], 0, 0, 0);
        }
      }
  };

  // ---------------------------------------------------------------- K loop
  // a sub-step's reads go out between its MFMAs
  auto order = [] {
    constexpr int kReads = TP * (kTP ? 2 : 1) + TQ * (kTQ ? 2 : 1), kMma = TP * TQ, kEach = (kReads + kMma - 1) / kMma;
#pragma unroll
    for (int i = 0; i < kMma; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, kEach, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // Two stages.  Fragments are read one sub-step ahead of their MFMAs.  Before the last sub-step's MFMAs a wave waits for
  // its loads of the next stage and its reads of this one; past the barrier the next stage is whole and this one free.
  // Stages past the last are loads of zeros that nothing reads: the loop stays one block, which the scheduler keeps as it
  // is written.
  if (steps > 0) {
    places(0);
    issue(0, 0);
    load_sf(0);
    places(1);
    store_sf(0, 0);
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    issue(1, 1);
    load_sf(1);
    places(2);
    read(0, 0, 0);
    read_sf(0);
    for (int ks = 0; ks < steps; ++ks) {
      const int buf = ks & 1;
      read(buf, 1, 1);
      mma(std::integral_constant<int, 0>{}, 0);
      order();
      read(buf, 2, 0);
      mma(std::integral_constant<int, 1>{}, 1);
      order();
      read(buf, 3, 1);
      mma(std::integral_constant<int, 2>{}, 0);
      order();
      store_sf(ks + 1, buf ^ 1);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      issue(ks + 2, buf);
      load_sf(ks + 2);
      places(ks + 3);
      read(buf ^ 1, 0, 0);
      mma(std::integral_constant<int, 3>{}, 1);
      __builtin_amdgcn_sched_barrier(0);
      read_sf(buf ^ 1);
    }
    __builtin_amdgcn_s_waitcnt(0);  // the loads of zeros have landed before the LDS is used again
  }

  // ---------------------------------------------------------------- output
  // Through LDS, as whole rows: a lane holds columns 8 v + 4 h .. + 4 of 32-column tile i, row r32 of 32-row tile j.
  constexpr int kEl = F32 ? 4 : 2, kLine = BP * kEl + 16;  // (padded: rows start in different banks)
  constexpr int kAtOnce = TL::kLds / kLine / 32 * 32 >= BQ ? BQ : TL::kLds / kLine / 32 * 32;
  static_assert(kAtOnce >= 32, "room for a slice of rows");
  for (int b = 0; b < BQ; b += kAtOnce) {
    if (q0 + b > q_last) break;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TQ; ++j) {
      const int row0 = (wq * TQ + j) * 32 - b;
      if (row0 < 0 || row0 >= kAtOnce) continue;
#pragma unroll
      for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint8_t* at = lds + (row0 + r32) * kLine + ((wp * TP + i) * 32 + 8 * v + 4 * h) * kEl;
          const f32x16& c = acc[i][j];
          if constexpr (F32)
            *(f32x4*)at = f32x4{c[4 * v], c[4 * v + 1], c[4 * v + 2], c[4 * v + 3]};
          else
            *(uint2*)at = uint2{bf16x2_rne(c[4 * v], c[4 * v + 1]), bf16x2_rne(c[4 * v + 2], c[4 * v + 3])};
        }
    }
    __syncthreads();
    constexpr int kLineChunks = BP * kEl / 16, kCols = 16 / kEl;
    for (int c = tid; c < kAtOnce * kLineChunks; c += kThreads) {
      const int row = c / kLineChunks, col = p0 + c % kLineChunks * kCols, q = q0 + b + row;
      if (q > q_last || b + row >= BQ || col >= p.p_cols) continue;
      i32x4 v = *(const i32x4*)(lds + row * kLine + c % kLineChunks * 16);
      long long to;
      if (WG) {
        to = (long long)t.expert * p.out_expert + (long long)q * p.out_ld;
      } else {
        int r = t.lo + q;
        if (p.out_pair) {
          r = p.src_info[r];
          if ((unsigned)r >= (unsigned)p.npairs) continue;
        }
        to = (long long)r * p.out_ld;
      }
      uint8_t* o = (uint8_t*)p.out + (to + col) * kEl;
      if constexpr (WG && F32) {
        if (p.accumulate) {
          const f32x4 sum = __builtin_bit_cast(f32x4, v) + *(const f32x4*)o;
          v = __builtin_bit_cast(i32x4, sum);
        }
      }
      *(i32x4*)o = v;
    }
  }
}

template <Op O, int BP, int BQ, int WP, int WQ, bool F32>
hipError_t launch_tile(GroupedParams& p, hipStream_t s) {
  p.p_tiles = (p.p_cols + BP - 1) / BP;
  long long grid;
  if (O == Op::WGRAD) {
    p.q_tiles = (p.q_cols + BQ - 1) / BQ;
    grid = (long long)p.E * p.q_tiles * p.p_tiles;
  } else {
    const long long groups = std::min(p.npairs, p.E);
    grid = (p.npairs + groups * (BQ - 1)) / BQ * p.p_tiles;
  }
  if (grid <= 0) return hipSuccess;
  grouped_kernel<O, BP, BQ, WP, WQ, F32, 8><<<dim3((unsigned)grid), dim3(64 * WP * WQ), 0, s>>>(p);
  return hipGetLastError();
}

Place place(Rows r, int T, int topk) {
  const bool whole = r != Rows::TOKEN || topk == 1;
  return Place{whole ? 0u : (uint32_t)(((1ull << 32) + topk - 1) / topk), whole ? -1 : 0, r == Rows::PLAN ? 0 : -1,
               r == Rows::TOKEN ? T : T * topk};
}

GroupedParams common(const GroupedArgs& a) {
  GroupedParams p{};
  p.start = a.start;
  p.src_info = a.src_info;
  p.E = a.E;
  p.npairs = a.T * a.topk;
  p.P = (const uint8_t*)a.w;
  p.Q = (const uint8_t*)a.a;
  p.K = a.k;
  p.p_cols = a.n;
  p.q_place = place(a.a_rows, a.T, a.topk);
  p.out = a.out;
  p.out_ld = a.n;
  p.out_pair = a.out_rows == Rows::PAIR;
  return p;
}

template <Op O, bool F32>
hipError_t launch_rows(GroupedParams& p, hipStream_t s) {
  return launch_tile<O, 256, 256, 4, 2, F32>(p, s);
}

// (the smallest tiles' extents)
constexpr int kMinP = 256, kMinQ = 256;

}  // namespace

bool grouped_gemm_fits(int npairs, int E, int n) {
  return (npairs / kMinQ + 1LL + std::min(npairs, E)) * ((n + kMinP - 1) / kMinP) < 0x7FFFFFFFLL;
}
bool grouped_wgrad_fits(int E, int n, int k) {
  return (long long)E * ((n + kMinQ - 1) / kMinQ) * ((k + kMinP - 1) / kMinP) < 0x7FFFFFFFLL;
}

hipError_t launch_grouped_gemm(const GroupedArgs& a, hipStream_t s) {
  GroupedParams p = common(a);
  p.p_expert = (long long)a.n * a.k * 2;
  p.p_ld = (a.w_kn ? a.n : a.k) * 2LL;
  p.q_ld = a.k * 2LL;
  if (a.w_kn) return a.out_f32 ? launch_rows<Op::GRAD, true>(p, s) : launch_rows<Op::GRAD, false>(p, s);
  return a.out_f32 ? launch_rows<Op::FWD, true>(p, s) : launch_rows<Op::FWD, false>(p, s);
}

hipError_t launch_grouped_gemm_mxfp4(const GroupedArgs& a, hipStream_t s) {
  GroupedParams p = common(a);
  p.p_expert = (long long)a.n * (a.k / 2);
  p.p_ld = p.q_ld = a.k / 2;
  p.sf_row = a.k / 32;
  p.p_sf_expert = (long long)a.n * p.sf_row;
  p.P_sf = (const uint8_t*)a.w_sf;
  p.Q_sf = (const uint8_t*)a.a_sf;
  return a.out_f32 ? launch_rows<Op::MX, true>(p, s) : launch_rows<Op::MX, false>(p, s);
}

hipError_t launch_grouped_wgrad(const WgradArgs& a, hipStream_t s) {
  GroupedParams p{};
  p.start = a.start;
  p.src_info = a.src_info;
  p.E = a.E;
  p.npairs = a.T * a.topk;
  p.P = (const uint8_t*)a.a;
  p.Q = (const uint8_t*)a.dout;
  p.p_ld = a.k * 2LL;
  p.q_ld = a.n * 2LL;
  p.p_cols = a.k;
  p.q_cols = a.n;
  p.p_place = place(a.a_rows, a.T, a.topk);
  p.q_place = place(a.dout_rows, a.T, a.topk);
  p.out = a.dw;
  p.out_ld = a.k;
  p.out_expert = (long long)a.n * a.k;
  p.accumulate = a.accumulate;
  return a.dw_f32 ? launch_tile<Op::WGRAD, 256, 256, 4, 2, true>(p, s)
                  : launch_tile<Op::WGRAD, 256, 256, 4, 2, false>(p, s);
}

}  // namespace moe
