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
#include <atomic>
#include <type_traits>

#include "gemm_common.h"
#include "grouped.h"
#include "tile_walk.h"

namespace moe {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned U32x2 __attribute__((ext_vector_type(2)));
typedef int i32x3 __attribute__((ext_vector_type(3)));

enum class Op { FWD, GRAD, WGRAD, MX };

// Where plan row r, pair src = src_info[r], lies in a tensor: at r, src or src / k.  (A quotient by a product is exact for
// src below 2^27, and there are at most 2^26 pairs: the error of ceil(2^32 / k) is below k <= 32.)
struct Place {
  uint32_t inverse;  // ceil(2^32 / k); 0: the pair itself
  int whole;         // -1: the pair itself, else 0
  int gathered;
  int places;        // the tensor's rows: a plan that is none reads nothing past them
  MOE_DEV int pair(int src) const { return (int)__umulhi((uint32_t)src, inverse) + (src & whole); }
  MOE_DEV int within(int at) const { return min(max(at, 0), places - 1); }
  MOE_DEV int of(int src) const { return within(pair(src)); }
  // the tensor's (below 4 GiB where it is gathered): what a tile's last columns would read past its last row is zeros
  MOE_DEV uint32_t bytes(uint32_t ld) const { return (uint32_t)places * ld; }
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
  long long p_sf_bytes, q_sf_bytes;
  int n_rows;            // MXFP4: weight rows of an expert
  uint32_t p_ld, q_ld;   // bytes between rows as they lie in memory
  int p_cols, q_cols;    // extents of the output (q_cols: WGRAD only, else the expert's rows)
  int K;                 // summed length (WGRAD: the expert's rows)
  int sf_row;            // MXFP4: K / 32
  Place q_place, p_place;
  uint8_t* out;
  uint32_t out_ld;       // bytes
  long long out_expert;  // WGRAD: bytes of one expert's dw
  int out_pair;          // rows go to src_info[r]
  int accumulate;
  int p_tiles, q_tiles;  // q_tiles: WGRAD only
  uint32_t p_inverse;    // floor(2^32 / p_tiles), of the kernels for few rows
};

// Direct-to-LDS loads: lane l's 16 (12) bytes land at l + 16 l; what lies out of the resource's bounds is zeros.
// Written so that the compiler does not see stores to LDS: it lets no ds_read_b64_tr pass one in flight.  The kernel's own
// waits order the two.  (m0 is no register that it keeps values in: it writes it right before what reads it, as here.
// Nor does it count the five states that have to pass between a vector instruction that writes a scalar register of the
// resource and such a load: settled() spends them where resources are made.  In the loads themselves they cost 1 %.)
constexpr uint32_t kAll = 0xFFFFF000u, kNone = kAll;  // the largest resource, an offset out of it (with what is added)
// (The offsets are the lanes' own: a scalar one may wrap the check against the resource's end, and the instruction's own
// would move the place in LDS with it.)
MOE_DEV void lds_copy16(i32x4 rsrc, uint32_t voff, uint32_t l) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(l), "v"(voff), "s"(rsrc)
               : "memory");
}
MOE_DEV void lds_copy12(i32x4 rsrc, uint32_t voff, uint32_t l) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx3 %1, %2, 0 offen lds" ::"s"(l), "v"(voff), "s"(rsrc)
               : "memory");
}
MOE_DEV uint32_t lds_address(const void* l) { return (uint32_t)(uintptr_t)(const LDS3 void*)l; }

// A value that is the same in every lane, in a scalar register.
MOE_DEV int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
// The same value, of which the compiler knows nothing: what follows from it is computed where it is used, not kept in
// registers through the K loop.
MOE_DEV int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}
MOE_DEV i32x4 settled(i32x4 rsrc) {
  asm volatile("s_nop 4" : "+s"(rsrc));
  return rsrc;
}
MOE_DEV i32x4 resource(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)base;
  return settled(i32x4{scalar((int)(uint32_t)b), scalar((int)(uint32_t)(b >> 32)), scalar((int)bytes), 0x00020000});
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

// start[e], made safe against a plan that is none.
MOE_DEV int row_at(const GroupedParams& p, int e) { return min(max(p.start[e], 0), p.npairs); }

// n / d, with inverse = floor(2^32 / d) for d > 1: at most one too small.
MOE_DEV int quotient(int n, int d, uint32_t inverse) {
  const int q = d == 1 ? n : (int)__umulhi((uint32_t)n, inverse);
  return q + (n - q * d >= d ? 1 : 0);
}

constexpr int kStream = 2;  // cache policy of stores: not kept

struct TileAt {
  bool ok;
  int expert, lo, hi;  // the expert's rows
  int q, p;            // tile indices within the expert
};

// The tiles of a workgroup, one after the other.  Tiles lie expert by expert, in groups of up to GQ q-tiles, within a group
// p-tile by p-tile, and each XCD takes a contiguous eighth, its workgroups in turn: what an XCD runs at once then shares few
// operand panels in its L2.  WGRAD, whose tiles cost what their expert has rows: an expert's tiles go in chunks of one for
// each workgroup of an XCD, the chunks to the XCDs in turn, so that an XCD's workgroups walk the same rows at the same time
// (an eighth of every expert's tiles for each XCD, whose workgroups then come apart, had an L2 hit rate of 45 %: 1889 us for
// 32 experts of 7168 x 2048 and 8192 tokens, with 74 % 1820); where that would leave workgroups without tiles, one after the other.
template <bool WGRAD, int BQ, int GQ>
struct Walk {
  int e0, before, upto;  // lane l: the tiles up to expert e0 + l's last
  int at, end, step, chunks;  // (WGRAD, chunks: at counts them)

  MOE_DEV void chunk(const GroupedParams& p, int first) {
    e0 = first;
    const int e = e0 + lane_id();
    int lo = 0, hi = 0;
    if (e < p.E) lo = row_at(p, e), hi = max(lo, row_at(p, e + 1));
    upto = before + wave_scan((hi - lo + BQ - 1) / BQ * p.p_tiles);
  }
  MOE_DEV void begin(const GroupedParams& p) {
    const int xcd = blockIdx.x & 7, in = blockIdx.x >> 3;
    step = gridDim.x >> 3;
    before = 0;
    if constexpr (WGRAD) {
      const int n = p.q_tiles * p.p_tiles;
      chunks = (n + step - 1) / step;
      if (chunks * step - n > n / 8) chunks = 0;
      at = chunks ? xcd : (int)blockIdx.x;
    } else {
      for (int e = 0;;) {
        chunk(p, e);
        e += 64;
        if (e >= p.E) break;
        before = __builtin_amdgcn_readlane(upto, 63);
      }
      const int G = __builtin_amdgcn_readlane(upto, 63), q = G >> 3, r = G & 7;
      at = xcd * q + min(xcd, r);
      end = at + q + (xcd < r ? 1 : 0);
      at += in;
      before = 0;
      if (p.E > 64) chunk(p, 0);
    }
  }
  MOE_DEV TileAt next(const GroupedParams& p) {
    TileAt t{};
    int within, q_tiles = p.q_tiles;
    if constexpr (WGRAD) {
      const int n = q_tiles * p.p_tiles;
      if (chunks) {
        for (;; at += 8) {
          t.expert = at / chunks;
          t.ok = t.expert < p.E;
          if (!t.ok) return t;
          const int c = at - t.expert * chunks;
          within = (int)((long long)n * c / chunks) + (blockIdx.x >> 3);
          if (within < (int)((long long)n * (c + 1) / chunks)) break;
        }
        at += 8 - step;
      } else {
        t.expert = at / n;
        t.ok = t.expert < p.E;
        if (!t.ok) return t;
        within = at - t.expert * n;
        at += (int)gridDim.x - step;
      }
      t.lo = row_at(p, t.expert);
      t.hi = max(t.lo, row_at(p, t.expert + 1));
    } else {
      t.ok = at < end;
      if (!t.ok) return t;
      while (at >= __builtin_amdgcn_readlane(upto, 63) && e0 + 64 < p.E)
        before = __builtin_amdgcn_readlane(upto, 63), chunk(p, e0 + 64);
      const unsigned long long later = __ballot(upto > at);
      if (!later) {  // (a plan that changed meanwhile)
        t.ok = false;
        return t;
      }
      const int l = __ffsll(later) - 1;
      t.expert = e0 + l;
      t.lo = row_at(p, t.expert);
      t.hi = max(t.lo, row_at(p, t.expert + 1));
      q_tiles = (t.hi - t.lo + BQ - 1) / BQ;
      within = at - (__builtin_amdgcn_readlane(upto, l) - q_tiles * p.p_tiles);
    }
    at += step;
    within = scalar(within);
    const TileIn in = tile_in(within, q_tiles, p.p_tiles, GQ);
    t.ok = in.ok;
    t.q = in.q;
    t.p = in.p;
    t.expert = scalar(t.expert);
    t.lo = scalar(t.lo);
    t.hi = scalar(t.hi);
    t.p = scalar(t.p);
    t.q = scalar(t.q);
    return t;
  }
};

// f(0), f(1) .. with the number as a type.
template <int FROM, int TO, class F>
MOE_DEV void each(F&& f) {
  if constexpr (FROM < TO) {
    f(std::integral_constant<int, FROM>{});
    each<FROM + 1, TO>(f);
  }
}

// Where 16-byte chunk c of row r lies among its row's eight (rows of 128 bytes).  A read serves lanes 0-7 together with
// 16-23: eight rows, and the two chunks that the lanes' second and third quarter differ by (bf16: 1, MXFP4: 2).
template <bool MX>
MOE_DEV int place_of_chunk(int c, int r) {
  return (MX ? (c & 4) | (c & 1) << 1 | (c >> 1 & 1) : c) ^ (r & 7);
}
template <bool MX>
MOE_DEV int chunk_at(int place, int r) {
  const int c = place ^ (r & 7);
  return MX ? (c & 4) | (c & 1) << 1 | (c >> 1 & 1) : c;
}

// Transposed operands: the 32-byte unit u of summed row r lies at u ^ trx(r), so that the 8 rows that 32 lanes read lie in
// different banks.
MOE_DEV int trx(int r) { return 2 * (r & 3) | (r >> 3 & 1); }

// ---------------------------------------------------------------- output
// From the registers.  In the plan's order nothing waits: the loads of the next tile are under way.  By pair the rows' src_info
// is loaded every 16 rows, and a sum that is added to (accumulate) ahead of every store; the wait for such a load covers the
// stores and the next tile's loads ahead of it (8192 tokens, 32 experts of 7168 x 2048: product 1557 us in the plan's order,
// 1615 by pair, MXFP4 621 and 678; weights' gradient in fp32 1806, accumulated 2181).  A lane holds columns 4 g .. + 4
// of row r16 of a 16 x 16 tile.  For bf16 two neighbouring tiles' lanes swap so that each has 8 in a row, and for both types
// lanes 8 apart then, so that a store is 8 rows of whole lines: 128 bytes.  Every store is issued, those out of the output
// with an offset that is dropped: the waits count them.
// A wave's tile from column p0 on, rows of them there; pair: they go to src_info[first ..], up to last.
template <int TP, int TQ, bool F32, bool WG>
MOE_DEV void store_tile(const GroupedParams& p, const f32x4 (&acc)[TP][TQ], const uint8_t* base, int p0, int rows, bool pair,
                        int first, int last) {
  constexpr int kEl = F32 ? 4 : 2, kTiles = F32 ? 2 : 4;  // kTiles tiles' columns are a line
  static_assert(TP % kTiles == 0, "lines");
  const __amdgpu_buffer_rsrc_t to = make_rsrc(base, pair ? kAll : (uint32_t)min(rows, TQ * 16) * p.out_ld);
  const int l = fresh(lane_id()), l16 = l & 15, lg = l >> 4, row8 = l16 & 7;
  // (past the last column: past the resource, with any row)
  constexpr uint32_t kPast = 0x80000000u;
  uint32_t column[TP / kTiles];
#pragma unroll
  for (int c = 0; c < TP / kTiles; ++c) {
    const int col = p0 + c * kTiles * 16 + (l16 >> 3) * (kTiles * 8) + (F32 ? 4 * lg : 16 * (lg & 1) + 8 * (lg >> 1));
    column[c] = col < p.p_cols ? (uint32_t)col * kEl : kPast;
  }
  uint32_t at[2] = {(uint32_t)row8 * p.out_ld, (uint32_t)(row8 + 8) * p.out_ld};
#pragma unroll
  for (int j = 0; j < TQ; ++j) {
    if (pair) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = j * 16 + h * 8 + row8, r = p.src_info[max(min(first + row, last), 0)];
        at[h] = row < rows && (uint32_t)r < (uint32_t)p.npairs ? (uint32_t)r * p.out_ld : kNone;
      }
    }
#pragma unroll
    for (int c = 0; c < TP / kTiles; ++c) {
      i32x4 d[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = c * kTiles + h * (kTiles / 2);
        if constexpr (F32) {
          d[h] = __builtin_bit_cast(i32x4, acc[i][j]);
        } else {
          const f32x4 u = acc[i][j], v = acc[i + 1][j];
          const auto x = __builtin_amdgcn_permlane16_swap(bf16x2_rne(u[0], u[1]), bf16x2_rne(v[0], v[1]), false, false);
          const auto y = __builtin_amdgcn_permlane16_swap(bf16x2_rne(u[2], u[3]), bf16x2_rne(v[2], v[3]), false, false);
          d[h] = i32x4{(int)x[0], (int)y[0], (int)x[1], (int)y[1]};
        }
      }
      i32x4 out[2];  // rows row8: lanes 8 .. 15 take the second half of lanes 0 .. 7's; rows row8 + 8: the other way round
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        out[0][e] = __builtin_amdgcn_update_dpp(d[0][e], d[1][e], 0x128, 0xF, 0xC, false);  // row_ror:8
        out[1][e] = __builtin_amdgcn_update_dpp(d[1][e], d[0][e], 0x128, 0xF, 0x3, false);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t o = at[h] + column[c];
        if (pair) o = at[h] == kNone || column[c] == kPast ? kNone : o;
        if constexpr (WG && F32) {
          if (p.accumulate) {
            const f32x4 sum = __builtin_bit_cast(f32x4, out[h]) +
                              __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(to, o, 0, 0));
            out[h] = __builtin_bit_cast(i32x4, sum);
          }
        }
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, out[h]), to, o, 0, kStream);
      }
    }
    at[0] += 16 * p.out_ld, at[1] += 16 * p.out_ld;
  }
}

// ---------------------------------------------------------------- tiles
// BP x BQ outputs, WP x WQ waves, each TP x TQ MFMA tiles of 16 x 16 (v_mfma_f32_16x16x32_bf16 and .._16x16x128_f8f6f4: the
// part's power limits a loop of MFMAs alone to 2.02 and 7.19 PFLOP/s with them, to 1.80 and 6.51 with the 32 x 32 forms).  A
// K-step (128 bytes of an operand's row) is staged in parts of 16 KB -- 128 rows, or columns, of P or Q -- in a ring of SLOTS
// of them.  Two tiles: 256 x 256, one workgroup a CU, whose operands cross LDS least often, and 128 x 128, two a CU.
template <Op O, int BP, int BQ, int WP, int WQ, int SLOTS>
struct GTile {
  static constexpr int kWaves = WP * WQ, kThreads = 64 * kWaves;
  static constexpr int TP = BP / 16 / WP, TQ = BQ / 16 / WQ;
  static constexpr bool kTP = O == Op::GRAD || O == Op::WGRAD, kTQ = O == Op::WGRAD;
  static constexpr int kPart = 16384, kPP = BP / 128, kPQ = BQ / 128, kParts = kPP + kPQ;
  static constexpr int kL = 16 / kWaves;  // a wave's loads of a part
  static constexpr int kSf = O == Op::MX ? (BP + BQ) * 16 : 0;  // scales: the words that hold a row's 8 (or two K-steps' 16)
  static constexpr int kLds = SLOTS * kPart + 2 * kSf;
  static constexpr int kBK = O == Op::MX ? 256 : 64;  // elements of a K-step
  static constexpr int kEarly = SLOTS - 2 * kParts;   // parts in flight past the next K-step's
  static_assert(BP % 128 == 0 && BQ % 128 == 0 && 128 % (TP * 16) == 0 && 128 % (TQ * 16) == 0, "a wave reads one part");
  static_assert(TP % 2 == 0 && TQ % 4 == 0 && TP <= TQ, "the order of reads");
  static_assert(16 % kWaves == 0 && kPP == kPQ && kEarly > 0 && kEarly <= kPP, "ring");
};

// WHERE: bit 0: P's rows, bit 1: Q's rows are found through src_info (WGRAD; elsewhere Q's are looked up once a tile); MX: bit
// 0: rows of scales are not whole words.
// Registers: one workgroup a CU for the large tile.
template <Op O, int BP, int BQ, int WP, int WQ, int SLOTS, bool F32, int WHERE>
__global__ __launch_bounds__(64 * WP * WQ, 2) void grouped_kernel(GroupedParams p) {
  using TL = GTile<O, BP, BQ, WP, WQ, SLOTS>;
  constexpr bool MX = O == Op::MX, WG = O == Op::WGRAD, kTP = TL::kTP, kTQ = TL::kTQ;
  constexpr int TP = TL::TP, TQ = TL::TQ, BK = TL::kBK, kThreads = TL::kThreads, L = TL::kL;
  constexpr int PT = TL::kParts, EARLY = TL::kEarly, LATE = PT - EARLY;
  __shared__ __attribute__((aligned(16))) uint8_t lds[TL::kLds];
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wave % WP, wq = wave / WP, g = lane >> 4, r16 = lane & 15;
  Walk<WG, BQ, 8> walk;
  walk.begin(p);
  TileAt now = walk.next(p);  // the tile of the MFMAs; the loads run up to two K-steps ahead, into `then`
  if (!now.ok) return;
  // (read in every trip: not to be loaded there again)
  const int total = scalar(p.K), sf_row = scalar(p.sf_row);
  auto steps_of = [&](const TileAt& t) { return max(2, ((WG ? t.hi - t.lo : total) + BK - 1) / BK); };

  // ---------------------------------------------------------------- what each lane loads
  // Load i of a part: rows (i * waves + wave) * 8 + lane / 8 of 128 bytes, or (T) summed rows (i * waves + wave) * 4 + lane
  // / 16 of 256 bytes.  Bases are scalar and move by a K-step, a lane's offsets stay until the last one.  Rows past the
  // last, of the output or summed, lie past the resource's end and chunks past K get an offset that does: both load zeros.
  // (Columns past a T operand's last are the next row's first; what comes of them is not stored.)
  constexpr int kStep8 = TL::kWaves * 8, kStep4 = TL::kWaves * 4;
  const int chunk8 = chunk_at<MX>(lane & 7, wave * 8 + (lane >> 3));
  constexpr bool kLookP = WG && (WHERE & 1), kLookQ = WG && (WHERE & 2);
  uint32_t p_off[kTP ? 1 : TL::kPP][L], q_off[kTQ ? 1 : TL::kPQ][L];  // (T: of part 0, the others lie 256 bytes on)
  i32x4 p_from{}, q_from{};      // the operands' resources at the next load's K-step
  int p_k = 0, q_k = 0;          // summed elements up to it
  int load_lo = 0, load_hi = 0;  // WGRAD: the rows of the loads' tile
  uint32_t p_skip = 0, q_skip = 0;  // T operands: bytes ahead of the tile's first column
  // the bytes of a T operand from its resource's base on: of a K-step
  auto t_extent = [&](bool isP) {
    const int left = (WG ? load_hi - load_lo : total) - (isP ? p_k : q_k);
    return left > 0 ? (uint32_t)min(left, 64) * (isP ? p.p_ld : p.q_ld) - (isP ? p_skip : q_skip) : 0u;
  };
  // the offset of a T operand's row and column of a part's first load
  auto t_off = [&](uint32_t ld) {
    const int l = fresh(lane), row = wave * 4 + (l >> 4);
    return (uint32_t)row * ld + ((((l & 15) >> 1) ^ trx(row)) << 5) + (l & 1) * 16;
  };
  // src_info of this lane's rows r0 + lane / (64 / N), by scalar loads: a vector load would have to wait for the loads into
  // LDS behind it
  auto source = [&](auto lanes, int r0, int last) {
    constexpr int N = decltype(lanes)::value;
    typedef const __attribute__((address_space(4))) int* Uniform;
    int v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = ((Uniform)(uintptr_t)p.src_info)[max(min(r0 + j, last), 0)];
    const int at = fresh(lane) / (64 / N);
    int r = v[0];
#pragma unroll
    for (int j = 1; j < N; ++j) r = at == j ? v[j] : r;
    return r;
  };
  auto aim_p = [&](const TileAt& t) {
    p_k = 0;
    p_skip = t.p * BP * 2;
    const uint8_t* base = p.P + (kTP ? (long long)p_skip : (long long)t.p * BP * p.p_ld);
    if constexpr (WG) {
      load_lo = t.lo, load_hi = t.ok ? t.hi : t.lo;
      base += kLookP ? 0 : (long long)t.lo * p.p_ld;
    } else {
      base += t.expert * p.p_expert;
    }
    const uint32_t off = kTP ? t_off(p.p_ld) : (uint32_t)(wave * 8 + (fresh(lane) >> 3)) * p.p_ld + chunk8 * 16;
#pragma unroll
    for (int j = 0; j < (kTP ? 1 : TL::kPP); ++j)
#pragma unroll
      for (int i = 0; i < L; ++i) p_off[j][i] = off + (kTP ? i * kStep4 : j * 128 + i * kStep8) * p.p_ld;
    p_from = resource(base, !t.ok    ? 0u
                            : kLookP ? p.p_place.bytes(p.p_ld) - p_skip
                            : kTP    ? t_extent(true)
                                     : (uint32_t)min(p.p_cols - t.p * BP, BP) * p.p_ld);
  };
  auto aim_q = [&](const TileAt& t) {
    q_k = 0;
    q_skip = t.q * BQ * 2;
    const uint8_t* base = p.Q + (kTQ ? (long long)q_skip : 0);
    const bool look = !WG && p.q_place.gathered;
    const int rows = t.hi - t.lo - t.q * BQ;
    if constexpr (WG)
      base += kLookQ ? 0 : (long long)t.lo * p.q_ld;
    else if (!look)
      base += ((long long)t.lo + t.q * BQ) * p.q_ld;
    const uint32_t off = kTQ ? t_off(p.q_ld) : (uint32_t)(wave * 8 + (fresh(lane) >> 3)) * p.q_ld + chunk8 * 16;
#pragma unroll
    for (int j = 0; j < (kTQ ? 1 : TL::kPQ); ++j)
#pragma unroll
      for (int i = 0; i < L; ++i) {
        q_off[j][i] = off + (kTQ ? i * kStep4 : j * 128 + i * kStep8) * p.q_ld;
        if (look && t.ok) {
          const int first = t.lo + t.q * BQ;
          q_off[j][i] = (uint32_t)p.q_place.of(source(std::integral_constant<int, 8>{}, first + j * 128 + i * kStep8 + wave * 8,
                                                      first + rows - 1)) * p.q_ld + chunk8 * 16;
        }
      }
    q_from = resource(base, !t.ok            ? 0u
                            : kLookQ || look ? p.q_place.bytes(p.q_ld) - (kTQ ? q_skip : 0)
                            : kTQ            ? t_extent(false)
                                             : (uint32_t)min(rows, BQ) * p.q_ld);
  };
  // WGRAD: the offsets of a K-step's rows through src_info (read also where only one operand's rows are found there).  Lane l
  // of src[v] holds that of this wave's row l % (4 L) of the tile's K-step kEach v + l / (4 L): a vector load, which has to wait
  // for the loads into LDS behind it, for 4 kEach K-steps, and a shuffle for each.  In pieces, which go between MFMAs.
  constexpr int kSrc = 4, kEach = 16 / L;
  int src[kSrc] = {}, src_k = 0, row[L] = {}, p_row[L] = {}, q_row[L] = {};
  uint32_t p_next[L] = {}, q_next[L] = {}, t_column = 0;
  if constexpr (kLookP || kLookQ) t_column = t_off(0);
  auto sources = [&](int k0) {  // of the K-steps from row k0 on
    if constexpr (kLookP || kLookQ) {
      const int l = fresh(lane), first = load_lo + k0 + l / (4 * L) * BK + (l >> 2) % L * kStep4 + wave * 4 + (l & 3);
      src_k = 0;
#pragma unroll
      for (int v = 0; v < kSrc; ++v) src[v] = p.src_info[max(min(first + v * kEach * BK, load_hi - 1), 0)];
#pragma unroll
      for (int v = 0; v < kSrc; ++v) asm volatile("" : "+v"(src[v]));  // (waits here, not in every trip)
    }
  };
  auto next_source = [&](int k0) {  // to the K-step at row k0
    if constexpr (kLookP || kLookQ) {
      if (++src_k % kEach == 0) {
        if (src_k == kEach * kSrc) {
          sources(k0);
        } else {
#pragma unroll
          for (int v = 1; v < kSrc; ++v) src[v - 1] = src[v];
        }
      }
    }
  };
  constexpr int kPieces = kLookP || kLookQ ? 6 : 0;
  auto piece = [&](int n, int k0) {  // of the offsets of the K-step at row k0
#pragma unroll
    for (int i = 0; i < L; ++i) {
      if (n == 0) {
        row[i] = __builtin_amdgcn_ds_bpermute((src_k % kEach * (4 * L) + i * 4 + g) * 4, src[0]);
      } else if (n == 1) {
        if constexpr (kLookP) p_row[i] = p.p_place.pair(row[i]);
        if constexpr (kLookQ) q_row[i] = p.q_place.pair(row[i]);
      } else if (n == 2) {
        if constexpr (kLookP) p_row[i] = p.p_place.within(p_row[i]);
        if constexpr (kLookQ) q_row[i] = p.q_place.within(q_row[i]);
      } else if (n == 3) {
        if constexpr (kLookP) p_next[i] = (uint32_t)p_row[i] * p.p_ld;
      } else if (n == 4) {
        if constexpr (kLookQ) q_next[i] = (uint32_t)q_row[i] * p.q_ld;
      } else {
        const bool live = k0 + i * kStep4 + wave * 4 + g < load_hi - load_lo;
        if constexpr (kLookP) p_next[i] = live ? p_next[i] + t_column : kNone;
        if constexpr (kLookQ) q_next[i] = live ? q_next[i] + t_column : kNone;
      }
    }
  };
  auto take_offsets = [&] {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      if constexpr (kLookP) p_off[0][i] = p_next[i];
      if constexpr (kLookQ) q_off[0][i] = q_next[i];
    }
  };
  auto offsets_at = [&](int k0) {
#pragma unroll
    for (int n = 0; n < kPieces; ++n) piece(n, k0);
    take_offsets();
    next_source(k0 + BK);
  };
  // load i of part J (P's first) of the K-step that its operand has come to, into a slot (its offset in LDS)
  const uint32_t lds0 = lds_address(lds);
  auto issue = [&](auto part, int i, uint32_t slot) {
    constexpr int J = decltype(part)::value;
    constexpr bool isP = J < TL::kPP, tr = isP ? kTP : kTQ;
    constexpr int j = isP ? J : J - TL::kPP;
    const uint32_t l = slot + (i * TL::kWaves + wave) * 1024;
    if constexpr (isP)
      lds_copy16(p_from, p_off[tr ? 0 : j][i] + (tr ? j * 256 : 0), l);
    else
      lds_copy16(q_from, q_off[tr ? 0 : j][i] + (tr ? j * 256 : 0), l);
  };
  // an operand's next K-step; the last one's masks (what lies past a tile's rows does so at every K-step)
  auto advance = [&](i32x4& from, bool isP) {
    (isP ? p_k : q_k) += BK;
    if (isP ? kLookP : kLookQ) return;
    const uint32_t by = (isP ? kTP : kTQ) ? 64 * (isP ? p.p_ld : p.q_ld) : 128;
    const uint32_t lo = (uint32_t)from[0] + by;
    from[1] = scalar(from[1] + (lo < by ? 1 : 0));
    from[0] = scalar((int)lo);
  };
  auto tail = [&](bool isP) {
    const bool tr = isP ? kTP : kTQ;
    const int k0 = isP ? p_k : q_k, K = WG ? load_hi - load_lo : total;
    if ((isP ? kLookP : kLookQ) || k0 + BK <= K) return;
    if (tr) {
      i32x4& from = isP ? p_from : q_from;
      if (from[2]) from = settled(i32x4{from[0], from[1], scalar((int)t_extent(isP)), from[3]});
    } else {
      const bool none = k0 + chunk8 * (MX ? 32 : 8) >= K;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        if (isP) {
          for (auto& off : p_off) off[i] = none ? kNone : off[i];
        } else {
          for (auto& off : q_off) off[i] = none ? kNone : off[i];
        }
      }
    }
  };

  // MXFP4: the words that hold a row's 8 scales of a K-step, waves 0 .. BP / 64 - 1 P's rows, the others Q's.  A row's scales
  // may start at any byte: the three words from the one that holds the first.
  static_assert(!MX || (BP + BQ == kThreads && BP % 64 == 0), "a thread for each row of scales");
  i32x4 sf_from{};
  uint32_t sf_off = 0;
  int sf_k = 0;                             // scales of a row up to the K-step that is read next
  // where the fragments' rows start in their words, bytes (rows 16 apart start alike)
  constexpr bool ODD = MX && (WHERE & 1);  // rows of scales are not whole words
  uint32_t p_shift = 0, q_shift[ODD ? TQ : 1] = {};
  // the row of p or q (of the tile) whose scales row's are, in its tensor
  auto sf_row_p = [&](const TileAt& t, int row) { return (long long)t.expert * p.n_rows + min(t.p * BP + row, p.p_cols - 1); };
  auto sf_row_q = [&](const TileAt& t, int row) {
    int r = max(min(t.lo + t.q * BQ + row, t.hi - 1), t.lo);
    if (p.q_place.gathered && t.ok) r = p.q_place.of(p.src_info[r]);
    return (long long)r;
  };
  auto aim_sf = [&](const TileAt& t) {
    if constexpr (MX) {
      const bool isp = wave < BP / 64;
      const uint8_t* all = isp ? p.P_sf : p.Q_sf;
      // from the tile's first row on (gathered rows: from the tensor's first, which is below 4 GiB)
      long long first = isp ? sf_row_p(t, 0) : p.q_place.gathered ? 0 : sf_row_q(t, 0);
      const long long begin = first * sf_row & ~3LL, end = (isp ? p.p_sf_bytes : p.q_sf_bytes) + 3 & ~3LL;
      const long long row = isp ? sf_row_p(t, tid) : sf_row_q(t, tid - BP);
      sf_off = (uint32_t)((row * sf_row & ~3LL) - begin);
      sf_from = resource(all + begin, t.ok ? (uint32_t)min(end - begin, (long long)kAll) : 0u);
    }
  };
  auto aim_shifts = [&](const TileAt& t) {
    if constexpr (ODD) {
      p_shift = (uint32_t)((t.expert * (long long)p.n_rows + t.p * BP + r16) * sf_row) & 3;
#pragma unroll
      for (int j = 0; j < TQ; ++j) q_shift[j] = (uint32_t)(sf_row_q(t, (wq * TQ + j) * 16 + r16) * sf_row) & 3;
    }
  };
  // kSfSteps K-steps' at a time: whole words of two (every row is a request of its own, which cost as much as 100 cycles of
  // the loop for 64 of them)
  constexpr int kSfSteps = ODD ? 1 : 2;
  auto load_sf = [&](int buf) {
    if constexpr (MX) {
      const uint32_t to = lds0 + SLOTS * TL::kPart + buf * TL::kSf + wave * (64 * 16);
      if constexpr (ODD)
        lds_copy12(sf_from, sf_off, to);
      else
        lds_copy16(sf_from, sf_off, to);
      sf_off += 8 * kSfSteps;
    }
  };

  // ---------------------------------------------------------------- fragments
  constexpr int kRing = SLOTS * TL::kPart;
  auto wrap = [](int at) { return at >= kRing ? at - kRing : at; };
  i32x4 fp[2][TP], fq[TQ];  // (a Q fragment's registers take the next sub-step's as soon as its MFMAs are out)
  uint32_t sp[TP / 2] = {}, sq[TQ / 2] = {};
  const int t_row = 8 * g + (r16 >> 2);
  const uint32_t t_lane = t_row * 256 + (trx(t_row) << 5) + (lane & 3) * 8;
  // tile: of 16 rows (columns) within the part at base
  auto frag = [&](const uint8_t* base, bool tr, int tile, int s) -> i32x4 {
    if (!tr)
      return *(const i32x4*)(base + (tile * 16 + r16) * 128 + place_of_chunk<MX>(MX ? 2 * g + s : 4 * s + g, r16) * 16);
    // (an exclusive or of an address that changes with the K-step, not a sum with one of a register a tile)
    const uint32_t a = (lds_address(base) + t_lane + s * (32 * 256)) ^ (uint32_t)(tile << 5);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS3 s16x4*)a);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS3 s16x4*)(a + 4 * 256));
    return __builtin_bit_cast(i32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  constexpr int kPw = 128 / (TP * 16), kQw = 128 / (TQ * 16);  // waves that share a part
  // a fragment of a sub-step of the K-step whose parts this wave reads lie at bp and bq
  auto read_p = [&](int i, int bp, int s) { fp[s & 1][i] = frag(lds + bp, kTP, wp % kPw * TP + i, s); };
  auto read_q = [&](int j, int bq, int s) { fq[j] = frag(lds + bq, kTQ, wq % kQw * TQ + j, s); };
  // a K-step's scales: lane g's blocks are 2 g and 2 g + 1, for sub-steps 0 and 1 (blocks past K: scale 2^-127, on codes of
  // zero)
  typedef uint16_t U16x2 __attribute__((ext_vector_type(2)));
  U16x2 sp_next[TP / 2] = {}, sq_next[TQ / 2] = {};  // two tiles' in a word
  auto read_sf = [&](int buf, int half) {
    if constexpr (MX) {
      typedef uint16_t __attribute__((aligned(1))) Anywhere;
      typedef std::conditional_t<ODD, Anywhere, uint16_t> Bytes2;
      const uint8_t* f = lds + SLOTS * TL::kPart + buf * TL::kSf + half * 8 + 2 * g + r16 * 16;
#pragma unroll
      for (int i = 0; i < TP; ++i) sp_next[i / 2][i % 2] = *(const Bytes2*)(f + (wp * TP + i) * 256 + p_shift);
#pragma unroll
      for (int j = 0; j < TQ; ++j)
        sq_next[j / 2][j % 2] = *(const Bytes2*)(f + (BP + (wq * TQ + j) * 16) * 16 + (ODD ? q_shift[j] : 0));
    }
  };
  auto take_sf = [&] {
    if constexpr (MX) {
#pragma unroll
      for (int i = 0; i < TP / 2; ++i) sp[i] = __builtin_bit_cast(uint32_t, sp_next[i]);
#pragma unroll
      for (int j = 0; j < TQ / 2; ++j) sq[j] = __builtin_bit_cast(uint32_t, sq_next[j]);
      sf_k += 8;
      if (sf_k > sf_row) {
        const int left = sf_row - sf_k + 8 - 2 * g;
        const uint32_t keep = left >= 2 ? 0xFFFFFFFFu : left == 1 ? 0x00FF00FFu : 0u;
#pragma unroll
        for (auto& word : sp) word &= keep;
#pragma unroll
        for (auto& word : sq) word &= keep;
      }
    }
  };
  f32x4 acc[TP][TQ];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
      for (int j = 0; j < TQ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  clear();
  auto mma = [&](auto sub, auto place) {
    constexpr int S = decltype(sub)::value, j = decltype(place)::value / TP, at = decltype(place)::value % TP;
    constexpr int i = j % 2 ? TP - 1 - at : at;  // (there and back: one operand of two stays, which takes less power)
    if constexpr (MX) {
      const i32x4 a = fp[S][i], b = fq[j];
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0}, i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, acc[i][j], 4, 4,
          S + 2 * (i & 1), (int)sp[i / 2], S + 2 * (j & 1), (int)sq[j / 2]);
    } else {
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fp[S][i]),
                                                          __builtin_bit_cast(bf16x8, fq[j]), acc[i][j], 0, 0, 0);
    }
  };

  constexpr int kStores = TP * TQ / (F32 ? 1 : 2);
  auto store = [&](const TileAt& t) {
    const int q0 = t.q * BQ + wq * TQ * 16, p0 = t.p * BP + wp * TP * 16;
    const bool pair = !WG && p.out_pair;
    const uint8_t* base = p.out;
    if (WG)
      base += t.expert * p.out_expert + (long long)q0 * p.out_ld;
    else if (!pair)
      base += ((long long)t.lo + q0) * p.out_ld;
    store_tile<TP, TQ, F32, WG>(p, acc, base, p0, max((WG ? p.q_cols : t.hi - t.lo) - q0, 0), pair, t.lo + q0, t.hi - 1);
  };

  // ---------------------------------------------------------------- K loop
  // A trip is a K-step: two sub-steps of TQ groups of TP MFMAs, with what else goes out between them.  (A wave that issues
  // many loads at once waits for the address unit, 16 cycles each and shared by the waves, and feeds no MFMAs meanwhile.)
  //   sub-step 0: the reads of sub-step 1's fragments, and the loads of the first parts of the K-step two ahead (as many as the
  //   ring has slots beside two K-steps')
  //   the first groups of sub-step 1; then the wait for the next K-step's loads and these reads, and the barrier: the next K-step
  //   is whole, and this one's slots are free
  //   the rest of sub-step 1: the reads of the next K-step's first fragments, and the loads of the other parts
  // The parts of the ring go out in order, each into the slot of the part SLOTS ahead of it.  A workgroup goes through its
  // tiles without draining the ring: the loads change to the next tile two K-steps ahead of the MFMAs (every tile has at
  // least two K-steps, of zeros past its last), past the last tile they are of zeros.  The order stays as it is written
  // (sched_barrier, and the accumulators pinned ahead of branches).
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  constexpr int kMma = TP * TQ, kGroups = TQ / 4, kBar = kGroups * TP;  // MFMAs of a sub-step, of sub-step 1 ahead of the barrier
  // load n of the parts FIRST .. behind the trip's first, whose slots are at[]
  auto issue_nth = [&](auto first, auto nth, const auto& at) {
    constexpr int n = decltype(nth)::value, part = decltype(first)::value + n / L;
    issue(std::integral_constant<int, part % PT>{}, n % L, at[n / L]);
    // (the operand's last part of the K-step)
    if (n % L == L - 1 && part % PT == TL::kPP - 1) advance(p_from, true);
    if (n % L == L - 1 && part % PT == PT - 1) advance(q_from, false);
  };
  auto pin = [&] {
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
      for (int j = 0; j < TQ; ++j) asm volatile("" : "+v"(acc[i][j]));
  };
  int steps = steps_of(now), ks = 0, slot = 0, buf = 0;  // (buf: of the scales that are read next)
  aim_p(now);
  aim_q(now);
  aim_sf(now);
  aim_shifts(now);
  load_sf(0);
  each<0, 2 * PT>([&](auto nth) {
    constexpr int n = decltype(nth)::value;
    if (n == 0) sources(0);
    if (n % PT == 0) offsets_at(n / PT * BK), tail(true);
    if (n % PT == TL::kPP) tail(false);
#pragma unroll
    for (int i = 0; i < L; ++i) issue(std::integral_constant<int, n % PT>{}, i, lds0 + n * TL::kPart);
    if (n % PT == TL::kPP - 1) advance(p_from, true);
    if (n % PT == PT - 1) advance(q_from, false);
  });
  if (kSfSteps == 1) load_sf(1);
  offsets_at(2 * BK);
  __builtin_amdgcn_s_waitcnt(0);
  __builtin_amdgcn_s_barrier();
  auto part_p = [&](int slot) { return wrap(slot + wp / kPw * TL::kPart); };
  auto part_q = [&](int slot) { return wrap(slot + (TL::kPP + wq / kQw) * TL::kPart); };
  int bp = part_p(0), bq = part_q(0);
#pragma unroll
  for (int i = 0; i < TP; ++i) read_p(i, bp, 0);
#pragma unroll
  for (int j = 0; j < TQ; ++j) read_q(j, bq, 0);
  read_sf(0, 0);
  TileAt then{};
  bool stored = false;
  for (;;) {
    const int next = wrap(slot + PT * TL::kPart);
    const bool change = ks == steps - 2;
    if (change) {
      then = walk.next(p);
      aim_p(then);
      aim_q(then);
      sources(0);
      offsets_at(0);
    }
    tail(true);
    tail(false);
    uint32_t early[EARLY], late[LATE];  // slots of the parts that go out ahead of the barrier and behind it
#pragma unroll
    for (int j = 0; j < EARLY; ++j) early[j] = scalar((int)(lds0 + wrap(slot + (2 * PT + j) * TL::kPart)));
#pragma unroll
    for (int j = 0; j < LATE; ++j)
      late[j] = scalar((int)(lds0 + slot + j * TL::kPart - (slot + j * TL::kPart >= kRing ? kRing : 0)));
    const int p_k_next = p_k + BK;  // of the loads of the next trip
    take_sf();
    each<0, kMma>([&](auto at) {
      constexpr int m = decltype(at)::value, kEvery = kMma / (EARLY * L);
      mma(I0{}, at);
      if (m < TP) read_p(m, bp, 1);
      if (m % TP == TP - 1) read_q(m / TP, bq, 1);
      if constexpr (m % kEvery == kEvery / 2)
        issue_nth(std::integral_constant<int, 2 * PT>{}, std::integral_constant<int, m / kEvery>{}, early);
      if constexpr (m % (kMma / 8) == 1 && m / (kMma / 8) < kPieces) piece(m / (kMma / 8), p_k_next);
      __builtin_amdgcn_sched_barrier(0);
    });
    each<0, kBar>([&](auto at) { mma(I1{}, at); });
    pin();
    next_source(p_k_next + BK);
    // (the stores of a tile that has just ended lie ahead of this trip's loads and may stay under way)
    if (stored)
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(EARLY * L + kStores));
    else
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(EARLY * L));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (change) aim_sf(then);
    // (the scales that are read next are the next tile's)
    if (ODD && ks == steps - 1) aim_shifts(then);
    const int ks_next = ks + 1 == steps ? 0 : ks + 1;
    if (ks_next % kSfSteps == 0) buf ^= 1;
    if (kSfSteps == 1 || change || (ks % kSfSteps == 0 && ks + 2 < steps)) load_sf(buf ^ 1);
    bp = part_p(next), bq = part_q(next);
    each<kBar, kMma>([&](auto at) {
      constexpr int m = decltype(at)::value, n = m - kBar, kEvery = (kMma - kBar) / (LATE * L);
      mma(I1{}, at);
      if (n < TP) read_p(n, bp, 0);
      if (n >= TP && n < TP + kGroups) read_q(n - TP, bq, 0);
      if (m % TP == TP - 1) read_q(m / TP, bq, 0);
      if constexpr (n % kEvery == kEvery / 2 && n / kEvery < LATE * L)
        issue_nth(std::integral_constant<int, SLOTS>{}, std::integral_constant<int, n / kEvery>{}, late);
      if (n == TP + kGroups) read_sf(buf, ks_next % kSfSteps);
      __builtin_amdgcn_sched_barrier(0);
    });
    take_offsets();
    slot = next;
    stored = ++ks == steps;
    if (stored) {
      store(now);
      if (!then.ok) break;
      now = then;
      steps = steps_of(now);
      ks = 0;
      sf_k = 0;
      clear();
    }
  }
  __builtin_amdgcn_s_waitcnt(0);  // the loads of zeros land before the workgroup's LDS is another's
}

// ---------------------------------------------------------------- few rows
// Where experts have few rows, the product is the weights' way through memory, and a tile of 256 rows spends its MFMAs and its
// loads on rows that are not there.  A workgroup takes 16 TP weight rows and 16 TQ rows of an expert; its W waves share the
// summed axis and read their parts straight from memory to the registers that the MFMAs take (a lane's 16 bytes lie side by
// side with three others': 64 bytes a row, and the line's other half comes with the wave's next load).  No wave waits for
// another until their sums meet in LDS, in the waves' order.  S loads of each row are under way: with 4 waves of one weight tile
// 4 tokens' product of 28672 x 4096 reads its active experts at 6.4 TB/s (two or four weight tiles a wave 5.1 and 5.6: fewer
// waves, less under way); MXFP4's rows, a quarter as long, go to two waves of two weight tiles (128 experts, 32 tokens: 5.4 TB/s,
// with one wave of one tile 5.3, with four 3.6).
template <bool MX, int TP, int TQ, int W, bool F32>
__global__ __launch_bounds__(64 * W, MX ? 2 : 4) void grouped_few_kernel(GroupedParams p) {
  constexpr int BQ = 16 * TQ, S = 8;
  __shared__ __attribute__((aligned(16))) float sums[W][BQ][16 * TP + 4];
  const int lane = lane_id(), wave = scalar((int)threadIdx.x >> 6), g = lane >> 4, r16 = lane & 15;
  // the workgroup's tile: q-tiles lie expert by expert, and each has all of its weight tiles in turn
  int slot = quotient((int)blockIdx.x, p.p_tiles, p.p_inverse);
  const int tile = (int)blockIdx.x - slot * p.p_tiles;
  int expert = -1, lo = 0, hi = 0;
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    const int e = e0 + lane;
    int from = 0, to = 0;
    if (e < p.E) from = row_at(p, e), to = max(from, row_at(p, e + 1));
    const int upto = wave_scan((to - from + BQ - 1) / BQ), all = __builtin_amdgcn_readlane(upto, 63);
    if (slot < all) {
      const int l = __ffsll((unsigned long long)__ballot(upto > slot)) - 1;
      expert = e0 + l;
      slot -= l ? __builtin_amdgcn_readlane(upto, l - 1) : 0;
      lo = __builtin_amdgcn_readlane(from, l) + slot * BQ;
      hi = __builtin_amdgcn_readlane(to, l);
      break;
    }
    slot -= all;
  }
  if (expert < 0) return;

  const int K = scalar((int)p.p_ld);  // bytes of a row
  const int p0 = tile * 16 * TP, p_rows = min(p.p_cols - p0, 16 * TP), rows = min(hi - lo, BQ);
  const bool look = p.q_place.gathered;
  const __amdgpu_buffer_rsrc_t from_p = make_rsrc(p.P + expert * p.p_expert + (long long)p0 * p.p_ld, (uint32_t)p_rows * p.p_ld);
  const __amdgpu_buffer_rsrc_t from_q =
      make_rsrc(p.Q + (look ? 0 : (long long)lo * p.q_ld), look ? p.q_place.bytes(p.q_ld) : (uint32_t)rows * p.q_ld);
  // the tensor's row of row r of the tile
  auto q_row = [&](int r) { return look ? p.q_place.of(p.src_info[min(lo + r, hi - 1)]) : min(r, rows - 1); };

  // A trip is S * 64 bytes of each row for each wave, in lines of kLine (MXFP4, for the scales' sake: all in one); load s is
  // 64 of them, at_load(s) bytes behind the first.
  constexpr int kLine = MX ? S * 64 : 128, kNext = S * 64 * W;
  auto at_load = [](int s) { return s * 64 / kLine * (kLine * W) + s * 64 % kLine; };
  int k = wave * kLine + g * 16;  // of the lane's next load
  uint32_t p_off[TP], q_off[TQ];
  i32x4 part[S][TP + TQ];
  auto load_p = [&](int s) {
#pragma unroll
    for (int i = 0; i < TP; ++i) part[s][i] = bload16(from_p, (k + at_load(s) < K ? p_off[i] : kNone) + at_load(s), 0);
  };
  int q_end[TQ];  // K, or 0 in rows that are not there
  auto load_q = [&](int s) {
#pragma unroll
    for (int j = 0; j < TQ; ++j) part[s][TP + j] = bload16(from_q, (k + at_load(s) < q_end[j] ? q_off[j] : kNone) + at_load(s), 0);
  };
  // MXFP4: a trip's 4 S scales of a row lie in four lanes, lane l having S of row l / 4: the words from the one that holds
  // the first, which the shift takes to the front.  The lane that multiplies block 4 s + g of row r16 has its word from lane
  // 4 r16 + (4 s + g) / S by a shuffle.  (A byte's load for each block took as long as the codes.)
  const int sf_lane = wave * (kLine / 16) + (lane & 3) * S;
  i32x3 sf_in[MX ? TP + TQ : 1];
  uint32_t sf[MX ? TP + TQ : 1][2], sf_off[MX ? TP + TQ : 1], sf_shift[MX ? TP + TQ : 1];
  const long long sfp0 = ((long long)expert * p.n_rows + p0) * p.sf_row & ~3LL, sfq0 = look ? 0 : (long long)lo * p.sf_row & ~3LL;
  const __amdgpu_buffer_rsrc_t from_psf =
      make_rsrc(p.P_sf + sfp0, (uint32_t)min((p.p_sf_bytes + 3 & ~3LL) - sfp0, (long long)kAll));
  const __amdgpu_buffer_rsrc_t from_qsf =
      make_rsrc(p.Q_sf + sfq0, (uint32_t)min((p.q_sf_bytes + 3 & ~3LL) - sfq0, (long long)kAll));
  auto aim_sf = [&](int i, long long row, long long first) {  // first: bytes of the tensor up to its resource
    const long long at = row * p.sf_row + sf_lane;
    sf_shift[i] = (uint32_t)at & 3;
    sf_off[i] = (uint32_t)((at & ~3LL) - first);
  };
  auto load_sf = [&](int i) {
    sf_in[i] = __builtin_bit_cast(i32x3, __builtin_amdgcn_raw_buffer_load_b96(i < TP ? from_psf : from_qsf, sf_off[i], 0, 0));
    sf_off[i] += kNext / 16;
  };
  auto take_sf = [&] {
    if constexpr (MX) {
#pragma unroll
      for (int i = 0; i < TP + TQ; ++i) {
        sf[i][0] = __builtin_amdgcn_alignbyte((uint32_t)sf_in[i][1], (uint32_t)sf_in[i][0], sf_shift[i]);
        sf[i][1] = __builtin_amdgcn_alignbyte((uint32_t)sf_in[i][2], (uint32_t)sf_in[i][1], sf_shift[i]);
      }
    }
  };
  auto scale = [&](int i, int s, bool in) {
    const uint32_t word = (uint32_t)__builtin_amdgcn_ds_bpermute((4 * r16 + s / 2) * 4, (int)sf[i][s % 2]);
    return (int)(in ? word >> 8 * g : 0u);
  };

#pragma unroll
  for (int i = 0; i < TP; ++i) {
    p_off[i] = (uint32_t)(i * 16 + r16) * p.p_ld + k;
    if constexpr (MX) aim_sf(i, (long long)expert * p.n_rows + p0 + i * 16 + (lane >> 2), sfp0), load_sf(i);
  }
  int source[TQ], source_sf[TQ];
#pragma unroll
  for (int j = 0; j < TQ; ++j) {
    source[j] = q_row(j * 16 + r16);
    if constexpr (MX) source_sf[j] = q_row(j * 16 + (lane >> 2));
  }
#pragma unroll
  for (int s = 0; s < S; ++s) load_p(s);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 0; j < TQ; ++j) {
    q_off[j] = (uint32_t)source[j] * p.q_ld + k;
    q_end[j] = j * 16 + r16 < rows ? K : 0;
    if constexpr (MX) aim_sf(TP + j, source_sf[j] + (look ? 0 : lo), sfq0), load_sf(TP + j);
  }
#pragma unroll
  for (int s = 0; s < S; ++s) load_q(s);
  f32x4 acc[TP][TQ];
#pragma unroll
  for (int i = 0; i < TP; ++i)
#pragma unroll
    for (int j = 0; j < TQ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto mma = [&](int s, int k) {
    int scales[MX ? TP + TQ : 1];
    if constexpr (MX) {
#pragma unroll
      for (int i = 0; i < TP + TQ; ++i) scales[i] = scale(i, s, k + at_load(s) < K);
    }
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
      for (int j = 0; j < TQ; ++j) {
        const i32x4 a = part[s][i], b = part[s][TP + j];
        if constexpr (MX)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0}, i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, acc[i][j], 4, 4, 0,
              scales[i], 0, scales[TP + j]);
        else
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                              acc[i][j], 0, 0, 0);
      }
  };
  for (int k0 = wave * kLine;;) {  // (the same in every lane)
    k0 += kNext;
    if (k0 >= K) break;
    take_sf();
    k += kNext;
#pragma unroll
    for (int i = 0; i < TP; ++i) p_off[i] += kNext;
#pragma unroll
    for (int j = 0; j < TQ; ++j) q_off[j] += kNext;
    if constexpr (MX) {
#pragma unroll
      for (int i = 0; i < TP + TQ; ++i) load_sf(i);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      mma(s, k - kNext);
      load_p(s);
      load_q(s);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  take_sf();
#pragma unroll
  for (int s = 0; s < S; ++s) mma(s, k);

  // a lane holds columns 4 g .. + 4 of row r16
#pragma unroll
  for (int i = 0; i < TP; ++i)
#pragma unroll
    for (int j = 0; j < TQ; ++j) *(f32x4*)&sums[wave][j * 16 + r16][i * 16 + 4 * g] = acc[i][j];
  __syncthreads();
  constexpr int kFours = 4 * TP;  // of a row
  const uint8_t* base = p.out + (p.out_pair ? 0 : (long long)lo * p.out_ld);
  const __amdgpu_buffer_rsrc_t to = make_rsrc(base, kAll);
  for (int n = threadIdx.x; n < BQ * kFours; n += 64 * W) {
    const int row = n / kFours, col = n % kFours * 4;
    f32x4 sum = *(const f32x4*)&sums[0][row][col];
#pragma unroll
    for (int w = 1; w < W; ++w) sum += *(const f32x4*)&sums[w][row][col];
    bool ok = row < rows && col < p_rows;
    uint32_t at = (uint32_t)row;
    if (p.out_pair && ok) {
      at = (uint32_t)p.src_info[lo + row];
      ok = at < (uint32_t)p.npairs;
    }
    const uint32_t o = ok ? at * p.out_ld + (uint32_t)(p0 + col) * (F32 ? 4 : 2) : kNone;
    if constexpr (F32)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sum), to, o, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b64(U32x2{bf16x2_rne(sum[0], sum[1]), bf16x2_rne(sum[2], sum[3])}, to, o, 0, 0);
  }
}

// ---------------------------------------------------------------- weight gradients of few rows
// With few rows an expert its gradient is written, not computed: a workgroup takes 128 x 128 of it, reads 64 rows of both
// operands at a time into LDS, and ends with its stores on their way; others of the compute unit's four load meanwhile.  (513
// tokens' gradients of 128 experts of 5760 x 2880, 16 rows each, bf16: 725 us, 5.9 TB/s; with the tiles above 985, whose next
// tile waits for the stores.)
template <bool F32, int WHERE>
__global__ __launch_bounds__(256, 4) void grouped_wgrad_few_kernel(GroupedParams p) {
  constexpr int kPart = 64 * 256, TP = 4, TQ = 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kPart];
  const int lane = lane_id(), wave = scalar((int)threadIdx.x >> 6), g = lane >> 4, r16 = lane & 15;
  const int up = quotient((int)blockIdx.x, p.p_tiles, p.p_inverse), tp = (int)blockIdx.x - up * p.p_tiles;
  const int expert = up / p.q_tiles, tq = up - expert * p.q_tiles;
  const int lo = scalar(row_at(p, expert)), hi = max(lo, scalar(row_at(p, expert + 1)));
  const uint32_t lds0 = lds_address(lds);
  f32x4 acc[TP][TQ];
#pragma unroll
  for (int i = 0; i < TP; ++i)
#pragma unroll
    for (int j = 0; j < TQ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int t_row = 8 * g + (r16 >> 2);
  const uint32_t t_lane = t_row * 256 + (trx(t_row) << 5) + (lane & 3) * 8;
  auto frag = [&](uint32_t part, int tile, int s) {
    const uint32_t a = (part + t_lane + s * (32 * 256)) ^ (uint32_t)(tile << 5);
    const s16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS3 s16x4*)a);
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS3 s16x4*)(a + 4 * 256));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  for (int k0 = lo; k0 < hi; k0 += 64) {
    const int subs = hi - k0 > 32 ? 2 : 1;
    const i32x4 from_p = resource(p.P + ((WHERE & 1) ? 0 : (long long)k0 * p.p_ld) + tp * 256, kAll);
    const i32x4 from_q = resource(p.Q + ((WHERE & 2) ? 0 : (long long)k0 * p.q_ld) + tq * 256, kAll);
    uint32_t p_off[4], q_off[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // rows 16 i + 4 wave + lane / 16
      const int l = i * 16 + wave * 4 + g, r = min(k0 + l, hi - 1), src = WHERE ? p.src_info[r] : 0;
      const uint32_t column = ((((uint32_t)r16 >> 1) ^ trx(wave * 4 + g)) << 5) + (r16 & 1) * 16;
      const bool in = k0 + l < hi;
      const uint32_t pr = (WHERE & 1) ? p.p_place.of(src) : r - k0, qr = (WHERE & 2) ? p.q_place.of(src) : r - k0;
      p_off[i] = in && tp * 256 + column < p.p_ld ? pr * p.p_ld + column : kNone;
      q_off[i] = in && tq * 256 + column < p.q_ld ? qr * p.q_ld + column : kNone;
    }
    if (k0 > lo) __syncthreads();  // (the rows before are read)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= 2 * subs) break;
      lds_copy16(from_p, p_off[i], lds0 + (i * 4 + wave) * 1024);
      lds_copy16(from_q, q_off[i], lds0 + kPart + (i * 4 + wave) * 1024);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    for (int s = 0; s < subs; ++s) {
      bf16x8 a[TP], b[TQ];
#pragma unroll
      for (int i = 0; i < TP; ++i) a[i] = frag(lds0, (wave & 1) * TP + i, s);
#pragma unroll
      for (int j = 0; j < TQ; ++j) b[j] = frag(lds0 + kPart, (wave >> 1) * TQ + j, s);
#pragma unroll
      for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int j = 0; j < TQ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    }
  }
  const int q0 = tq * 128 + (wave >> 1) * (TQ * 16);
  store_tile<TP, TQ, F32, true>(p, acc, p.out + expert * p.out_expert + (long long)q0 * p.out_ld, tp * 128 + (wave & 1) * (TP * 16),
                                max(p.q_cols - q0, 0), false, 0, 0);
}

// Compute units of the current device (cached per device).
int device_cus() {
  static std::atomic<int> cus[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
  int n = cus[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
    cus[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <Op O, int BP, int BQ, int WP, int WQ, int SLOTS, bool F32, int WHERE = 0>
hipError_t launch_tile(GroupedParams& p, hipStream_t s) {
  p.p_tiles = (p.p_cols + BP - 1) / BP;
  long long tiles;
  if (O == Op::WGRAD) {
    p.q_tiles = (p.q_cols + BQ - 1) / BQ;
    tiles = (long long)p.E * p.q_tiles * p.p_tiles;
  } else {
    const long long groups = std::min(p.npairs, p.E);
    tiles = (p.npairs + groups * (BQ - 1)) / BQ * p.p_tiles;
  }
  if (tiles <= 0) return hipSuccess;
  // one workgroup a CU walks its tiles; a multiple of the 8 XCDs
  const int per_cu = 163840 / GTile<O, BP, BQ, WP, WQ, SLOTS>::kLds, cus = std::max(8, device_cus() & ~7);
  const unsigned grid = (unsigned)std::min<long long>((tiles + 7) & ~7LL, (long long)cus * per_cu);
  grouped_kernel<O, BP, BQ, WP, WQ, SLOTS, F32, WHERE><<<dim3(grid), dim3(64 * WP * WQ), 0, s>>>(p);
  return hipGetLastError();
}

// grouped_few_kernel's workgroups
long long few_tiles(const GroupedParams& p, int TP, int TQ) {
  const long long groups = std::min(p.npairs, p.E), slots = (p.npairs + groups * (16 * TQ - 1)) / (16 * TQ);
  return slots * ((p.p_cols + 16 * TP - 1) / (16 * TP));
}
bool few_fits(const GroupedParams& p, int TP, int TQ, int W) { return few_tiles(p, TP, TQ) * 64 * W < 1LL << 32; }

template <bool MX, int TP, int TQ, int W, bool F32>
hipError_t launch_few(GroupedParams& p, hipStream_t s) {
  p.p_tiles = (p.p_cols + 16 * TP - 1) / (16 * TP);
  p.p_inverse = (uint32_t)((1ull << 32) / p.p_tiles);
  const long long tiles = few_tiles(p, TP, TQ);
  if (tiles == 0) return hipSuccess;
  grouped_few_kernel<MX, TP, TQ, W, F32><<<dim3((unsigned)tiles), dim3(64 * W), 0, s>>>(p);
  return hipGetLastError();
}

Place place(Rows r, int T, int topk) {
  const bool whole = r != Rows::TOKEN || topk == 1;
  return Place{whole ? 0u : (uint32_t)(((1ull << 32) + topk - 1) / topk), whole ? -1 : 0, r != Rows::PLAN,
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
  p.out = (uint8_t*)a.out;
  p.out_ld = (uint32_t)a.n * (a.out_f32 ? 4 : 2);
  p.out_pair = a.out_rows == Rows::PAIR;
  return p;
}

template <Op O, bool F32>
hipError_t launch_rows(GroupedParams& p, hipStream_t s) {
  // Rows of an expert that has any, on average, and the tiles that they make (masked slots count as rows: which they are only
  // the plan in device memory says).  us measured, by rows an expert:
  //   bf16, 8 experts of 28672 x 4096     1    4    8   16   64  128      MXFP4, 128 of 5760 x 2880    1    4    8   12   16   32
  //   grouped_few_kernel                198  320  364  552                32 x 16, 2 waves           134  206  238  265  307  444
  //   128 x 128                         245  327  330  340  352  495      32 x 32, 2 waves           162  242  260  273  286  387
  //   256 x 256                         290  421  427  426  439  447      256 x 256                  231  345  355  358  360  369
  // Where the tiles leave most of the part without work, the smaller ones are faster beyond that (bf16, 2 experts of 4096 x
  // 14336, 16 rows: 76 us, 128 x 128 143; MXFP4, 32 rows: 35, 256 x 256 89).
  const long long groups = std::max(1, std::min(p.npairs, p.E)), rows = (p.npairs + groups - 1) / groups;
  auto tiles = [&](int n) { return groups * ((p.p_cols + n - 1) / n) * ((rows + n - 1) / n); };
  const int cus = device_cus();
  if constexpr (O == Op::MX) {
    if (rows <= 12 && few_fits(p, 2, 1, 2)) return launch_few<true, 2, 1, 2, F32>(p, s);
    if ((rows <= 24 || (rows <= 128 && tiles(256) <= cus / 4)) && few_fits(p, 2, 2, 2))
      return launch_few<true, 2, 2, 2, F32>(p, s);
    return p.sf_row % 4 ? launch_tile<O, 256, 256, 4, 2, 9, F32, 1>(p, s) : launch_tile<O, 256, 256, 4, 2, 9, F32>(p, s);
  } else {
    if constexpr (O == Op::FWD)
      if ((rows <= 4 || (rows <= 32 && tiles(128) <= cus / 2)) && few_fits(p, 1, 1, 4))
        return launch_few<false, 1, 1, 4, F32>(p, s);
    if (rows <= 64 || tiles(256) < cus) return launch_tile<O, 128, 128, 2, 2, 5, F32>(p, s);
    return launch_tile<O, 256, 256, 4, 2, 10, F32>(p, s);
  }
}

template <bool F32, int WHERE>
hipError_t launch_wgrad(GroupedParams& p, hipStream_t s) {
  // Rows an expert, on average (us measured, 128 experts of 5760 x 2880; bf16: 16 rows 725, 48 805, 64 1112, with the large
  // tile 985, 991, 1036; fp32: 16 1574, 64 1585, 128 2097, with it 1594, 1657, 1822):
  const long long groups = std::max(1, std::min(p.npairs, p.E)), rows = (p.npairs + groups - 1) / groups;
  const long long tiles = (long long)p.E * ((p.p_cols + 127) / 128) * ((p.q_cols + 127) / 128);
  if (rows <= (F32 ? 64 : 48) && tiles * 256 < 1LL << 32) {
    p.p_tiles = (p.p_cols + 127) / 128;
    p.q_tiles = (p.q_cols + 127) / 128;
    p.p_inverse = (uint32_t)((1ull << 32) / p.p_tiles);
    grouped_wgrad_few_kernel<F32, WHERE><<<dim3((unsigned)tiles), dim3(256), 0, s>>>(p);
    return hipGetLastError();
  }
  // (16 experts of 512 x 512, 256 rows each: 11 us, with the large tile 20; from a tile a CU on the large one is as fast)
  if ((long long)p.E * ((p.p_cols + 255) / 256) * ((p.q_cols + 255) / 256) < device_cus())
    return launch_tile<Op::WGRAD, 128, 128, 2, 2, 5, F32, WHERE>(p, s);
  return launch_tile<Op::WGRAD, 256, 256, 4, 2, 10, F32, WHERE>(p, s);
}
template <bool F32>
hipError_t launch_wgrad(GroupedParams& p, hipStream_t s) {
  // (no rows: src_info is not read)
  switch (p.npairs == 0 ? 0 : (p.p_place.gathered ? 1 : 0) | (p.q_place.gathered ? 2 : 0)) {
    case 0: return launch_wgrad<F32, 0>(p, s);
    case 1: return launch_wgrad<F32, 1>(p, s);
    case 2: return launch_wgrad<F32, 2>(p, s);
    default: return launch_wgrad<F32, 3>(p, s);
  }
}

// (the smallest tiles' extents)
constexpr int kMinP = 128, kMinQ = 128;

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
  p.p_ld = (uint32_t)(a.w_kn ? a.n : a.k) * 2;
  p.q_ld = (uint32_t)a.k * 2;
  if (a.w_kn) return a.out_f32 ? launch_rows<Op::GRAD, true>(p, s) : launch_rows<Op::GRAD, false>(p, s);
  return a.out_f32 ? launch_rows<Op::FWD, true>(p, s) : launch_rows<Op::FWD, false>(p, s);
}

hipError_t launch_grouped_gemm_mxfp4(const GroupedArgs& a, hipStream_t s) {
  GroupedParams p = common(a);
  p.p_expert = (long long)a.n * (a.k / 2);
  p.p_ld = p.q_ld = (uint32_t)a.k / 2;
  p.sf_row = a.k / 32;
  p.n_rows = a.n;
  p.p_sf_bytes = (long long)a.E * a.n * p.sf_row;
  p.q_sf_bytes = (long long)(a.a_rows == Rows::TOKEN ? a.T : p.npairs) * p.sf_row;
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
  p.p_ld = (uint32_t)a.k * 2;
  p.q_ld = (uint32_t)a.n * 2;
  p.p_cols = a.k;
  p.q_cols = a.n;
  p.p_place = place(a.a_rows, a.T, a.topk);
  p.q_place = place(a.dout_rows, a.T, a.topk);
  p.out = (uint8_t*)a.dw;
  p.out_ld = (uint32_t)a.k * (a.dw_f32 ? 4 : 2);
  p.out_expert = (long long)a.n * p.out_ld;
  p.accumulate = a.accumulate;
  return a.dw_f32 ? launch_wgrad<true>(p, s) : launch_wgrad<false>(p, s);
}

}  // namespace moe
