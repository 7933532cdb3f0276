// Matrix product of two operands held in panels, Y[j, i] = sum_k A[i, k] B[j, k],
// shared by the 8-bit block-scaled product and the cross entropy.
//
// A panel is 16 rows; a step of a panel is 2 KiB: 128 columns of 8-bit codes
// or 64 columns of 16-bit values, in two halves of 1 KiB of four 256-byte
// units g of 16 bytes for each row r:
//   8 bits   half h, unit g, row r: columns 64 h + 16 g + 0..15 at 256 g + 16 r
//   16 bits  columns 32 h + 8 g + 0..7 at 256 g + 16 r
// Lane L of a wavefront takes row L%16 and unit L/16, which makes a half the
// operand of a 16x16x32 matrix instruction (16 bits) and two halves that of a
// 16x16x128 one (8 bits): a tile goes from memory to LDS as it lies and every
// LDS read is 64 lanes over 1 KiB without a bank conflict.  (Which columns a
// lane holds does not matter to the sum as long as both operands agree.)
// Panel p's steps are contiguous, at (p * steps + s) * 2048.
//
// A 16-bit operand may also be read the other way round, its columns as the
// product's rows and its rows as the summed index, with the transposing LDS
// read (ds_read_b64_tr_b16: of 16 lanes, lane 4 i + c points at the four
// columns 4 c.. of row i and lane j receives column j of rows 0..3).  On its
// way into LDS such an operand's rows 0..7 and 8..15 change places in odd
// units, which puts the eight 64-byte pieces of 32 lanes on different banks.
// (The straight read wants them in order: exchanged, its 1 KiB took 12 cycles
// instead of 8.)  A lane then holds, of the 32 rows of a
// half step, rows 16 (q/2) + 4 (q%2) + {0..3, 8..11}, q = L/16; where the other
// operand is read straight, its columns are stored in that order.
//
// An 8-bit weight may be read the other way round too, as a 16-bit operand: of
// 16 lanes, lane 2 i + c points at the eight codes 8 c.. of row i and lane j
// receives column j of rows 0..7 (ds_read_b64_tr_b8); a lane holds rows
// 16 (q/2) + 8 (q%2) + 0..7 of 32, and the codes are widened with their block's
// scale (one for the 64 rows of a step, which lie in one block of 128).
//
// 8-bit operands carry one exponent byte per row and step (E8M0: 2^(byte -
// 127)), four steps to a 32-bit word, word (s / 4) * scale_pitch + row; the
// matrix instruction takes the word of its lane's row as it is and multiplies
// the products of a step by both operands' powers of two.
#ifndef HYB_PANEL_H_
#define HYB_PANEL_H_

#include "hyb_device.h"

namespace hyb {
namespace {

typedef __attribute__((ext_vector_type(8))) int i32x8_t;
typedef __attribute__((ext_vector_type(4))) int srd4_t;

// Element kinds of a panel product beside HYB_F16 and HYB_BF16: 8-bit codes
// through the scaled 8-bit instruction, or widened (exactly) to bf16, scale
// included, for the 16-bit one.
//
// Why both.  The 8-bit instruction (the scaled form as well as the plain
// 16x16x32 one) does not sum its products to fp32 accuracy: over random codes
// of all exponents its result is off by up to 2^-11 of the largest product of
// the 128 (5e-5 of the result in the 2-norm); over products within a
// 15-bit window it is exact, so bits of a product far below the largest one
// are dropped.  The 16-bit instruction has no such loss, at half the rate.
// Outputs that keep fp32 take the wide kind, 16-bit outputs (whose rounding is
// 2^-8 or 2^-11 of the result) the fast one.
constexpr int kF8 = 0;
constexpr int kF8Wide = -1;
constexpr bool is_f8(int kind) { return kind <= 0; }

struct PanelOperand {
  const char* data;
  int32_t rows16;         // rows rounded up to 16 (the panels that exist)
  int32_t steps;          // steps per panel
  const uint32_t* scale;  // 8-bit operands only
  int64_t scale_pitch;    // words from four steps' scales to the next four's
  // Rows row0.. (a multiple of b1) of a packed matrix (hyb.h), whose tiles are
  // panels of their own (b1 / 16 of b2 / 64 steps): `data` is the dense stream,
  // where tile t lies in slot tidx[t] if that is one of n_dense; the other
  // tiles, and those of tile rows that reach beyond row `plain`, lie in
  // `spare`, tile rows spare0 .. spare1 - 1 (from row0) in the order of the
  // tiles; where it does not hold their row they read as zeros.
  int32_t log_b1, log_b2, tiles_k, n_dense;
  int64_t row0, plain;
  const int32_t* tidx;
  const char* spare;
  int32_t spare0, spare1;
  // An 8-bit weight read transposed: rows from `plain` on count as zeros; in
  // fp16 the values are divided by 2^(*top - 133).
  const uint32_t* top;
};

__device__ __forceinline__ srd4_t panel_srd(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return srd4_t{__builtin_amdgcn_readfirstlane(int(a & 0xFFFFFFFFu)),
                __builtin_amdgcn_readfirstlane(int((a >> 32) & 0xFFFFu)),
                __builtin_amdgcn_readfirstlane(int(bytes)), kBufDword3};
}

// 16 bytes per lane from srd + voffset into LDS at lds + 16 * lane; past the
// resource's end zeros are written.  Issued from inline assembly so that
// the compiler does not tie LDS reads to transfers of a later step; the
// caller waits (panel_wait) before its barrier.
__device__ __forceinline__ void panel_dma16(srd4_t srd, uint32_t lds, int voffset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voffset), "s"(srd)
               : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void panel_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t panel_lds_addr(const void* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) char*)(p)));
}

// Registers of one panel's step: as loaded, or widened to bf16.
template <int KIND>
struct PanelRegs {
  u32x4_t v[KIND == kF8Wide ? 4 : 2];
};

// The loaded halves of a step as operand registers; `scale` is the lane's
// scale word.  (v_cvt_scalef32_pk_bf16_fp8 reads only the exponent of its
// scale; 4 significant bits and a power of two are exact in bf16.)
template <int KIND, int BYTE>
__device__ __forceinline__ PanelRegs<KIND> panel_regs(u32x4_t h0, u32x4_t h1, uint32_t scale) {
  PanelRegs<KIND> r;
  if constexpr (KIND == kF8Wide) {
    const float f = __builtin_bit_cast(float, ((scale >> (8 * BYTE)) & 0xFFu) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(h0[i], f, false));
      r.v[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(h0[i], f, true));
      r.v[2 + (i >> 1)][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(h1[i], f, false));
      r.v[2 + (i >> 1)][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(h1[i], f, true));
    }
  } else {
    r.v[0] = h0;
    r.v[1] = h1;
  }
  return r;
}

// One step's product of a panel pair: 128 (8-bit) or 64 (16-bit) columns.
template <int KIND, int BYTE>
__device__ __forceinline__ f32x4_t panel_mfma(const PanelRegs<KIND>& ar, const PanelRegs<KIND>& br, f32x4_t c,
                                              uint32_t sa, uint32_t sb) {
  const auto& a = ar.v;
  const auto& b = br.v;
  if constexpr (KIND == kF8Wide) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = mfma16x16x32<HYB_BF16>(__builtin_bit_cast(uint4, a[i]), __builtin_bit_cast(uint4, b[i]), c);
    return c;
  } else if constexpr (KIND == kF8) {
    const i32x8_t av = {int(a[0][0]), int(a[0][1]), int(a[0][2]), int(a[0][3]),
                        int(a[1][0]), int(a[1][1]), int(a[1][2]), int(a[1][3])};
    const i32x8_t bv = {int(b[0][0]), int(b[0][1]), int(b[0][2]), int(b[0][3]),
                        int(b[1][0]), int(b[1][1]), int(b[1][2]), int(b[1][3])};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 0, 0, BYTE, int(sa), BYTE, int(sb));
  } else {
    c = mfma16x16x32<KIND>(__builtin_bit_cast(uint4, a[0]), __builtin_bit_cast(uint4, b[0]), c);
    return mfma16x16x32<KIND>(__builtin_bit_cast(uint4, a[1]), __builtin_bit_cast(uint4, b[1]), c);
  }
}

// 16 and 8 bytes at any 2-byte aligned address (the hardware takes unaligned
// global accesses).
struct __attribute__((packed, aligned(2))) Bytes16 {
  uint32_t w[4];
};
struct __attribute__((packed, aligned(2))) Bytes8 {
  uint32_t w[2];
};

// Two or four fp32 values to 16 bits, to nearest even: one instruction for two
// (rounding in integers takes six for each).
template <int DT>
__device__ __forceinline__ uint32_t round16x2(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) float f32x2_t;
  const f32x2_t v = {a, b};
  if constexpr (DT == HYB_BF16) {
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
  } else {
    typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
  }
}
template <int DT>
__device__ __forceinline__ uint2 round16x4(float a, float b, float c, float d) {
  return make_uint2(round16x2<DT>(a, b), round16x2<DT>(c, d));
}

// A wavefront's KA x KB panels of 16-bit results, row by row.  In registers a
// lane has four columns of a row, so a store would cover 32 bytes of each of
// 16 rows; through LDS (its own 512 KA KB bytes, 16-byte units rotated by the
// row against bank conflicts) 16-byte stores cover KA * 32 bytes of a row.
// quad(i, j) gives the four values of acc[i][j] as two words, row16 the lane's
// row of 16; put(row, column, values) stores eight columns.
template <int KA, int KB, typename Quad, typename Put>
__device__ __forceinline__ void panel_rows16(char* lds, int lane, int row16, Quad quad, Put put) {
  constexpr int kUnits = KA * 2;  // of a row
#pragma unroll
  for (int j = 0; j < KB; ++j)
#pragma unroll
    for (int i = 0; i < KA; ++i) {
      const int row = j * 16 + row16, unit = i * 2 + (lane >> 5);
      *reinterpret_cast<uint2*>(lds + row * (kUnits * 16) + ((unit ^ (row & (kUnits - 1))) * 16) + ((lane >> 4) & 1) * 8) =
          quad(i, j);
    }
  // one wavefront writes and reads its own part: its accesses done suffices
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  constexpr int kRows = 64 / kUnits;  // per store
#pragma unroll
  for (int r = 0; r < KB * 16; r += kRows) {
    const int row = r + lane / kUnits, unit = lane % kUnits;
    put(row, unit * 8, *reinterpret_cast<const uint4*>(lds + row * (kUnits * 16) + ((unit ^ (row & (kUnits - 1))) * 16)));
  }
}

// Workgroups run round-robin over the 8 XCDs (id L on XCD L % 8), each with
// its own L2.  XCD x takes a contiguous range of an order in which 4 A blocks
// are swept across all B blocks before the next 4, so workgroups that run
// together on one XCD share A and B panels in its L2.
__device__ __forceinline__ int32_t panel_order(int32_t id, int32_t total) {
  constexpr int32_t kXcd = 8;
  const int32_t xcd = id % kXcd, per = total / kXcd, extra = total % kXcd;
  return xcd * per + (xcd < extra ? xcd : extra) + id / kXcd;
}
__device__ __forceinline__ void panel_block(int32_t g, int32_t na, int32_t nb, int32_t& ab, int32_t& bb) {
  constexpr int32_t kGroup = 4;
  const int32_t first = g / (kGroup * nb) * kGroup;
  const int32_t width = na - first < kGroup ? na - first : kGroup;
  const int32_t r = g - first * nb;
  bb = r / width;
  ab = first + r % width;
}

typedef __attribute__((ext_vector_type(4))) short i16x4_t;
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;
typedef __attribute__((ext_vector_type(2))) int i32x2_t;
typedef __attribute__((address_space(3))) i32x2_t lds_i32x2_t;

// LDS-fed tile: AP x BP panels per workgroup of WA x WB wavefronts, STAGES LDS
// stages of one step each (transfers run STAGES - 1 steps ahead).  TA / TB:
// that operand is read transposed (its "panels" here are blocks of 16 of its
// columns).  TILED: A lies in tiles (PanelOperand).  CODES: A is an 8-bit weight
// read transposed by a 16-bit product.
template <int KIND, int AP, int BP, int WA, int WB, int STAGES = 2, bool TA = false, bool TB = false, bool TILED = false,
          bool CODES = false>
struct PanelTile {
  static_assert(STAGES == 2 || STAGES == 4, "a step's stage is an immediate of the loop unrolled by four");
  static constexpr int kWaves = WA * WB;
  static constexpr int kA = AP / WA, kB = BP / WB;  // panels per wavefront
  static constexpr int kStageA = CODES ? AP * 1024 : AP * 2048;
  static constexpr int kStage = kStageA + BP * 2048;
  static constexpr int kScaleStage = is_f8(KIND) ? (AP + BP) * 64 : 0;  // a word per row, four steps
  static constexpr int kLds = STAGES * kStage + 2 * kScaleStage;
  static constexpr int kLoadsA = (CODES ? AP : AP * 2) / kWaves, kLoadsB = BP * 2 / kWaves;  // 1 KiB transfers per wavefront and step
  static_assert(AP % WA == 0 && BP % WB == 0 && AP * 2 % kWaves == 0 && BP * 2 % kWaves == 0, "even split");
  static_assert(!(TA || TB) || !is_f8(KIND), "8-bit operands are read straight");

  // One operand's transfers of step s into its part of a stage.
  // (prepare() sets up a step, put() issues one of a wavefront's transfers.)
  template <bool T, int P, int LOADS>
  struct Feed {
    srd4_t rsrc;
    const char* data;
    int64_t pitch, total;
    int32_t first;

    // Straight: panels p0.., the resource ends with the last panel (panels
    // behind it read as zeros).  Transposed: columns 16 p0.. of all panels; a
    // step is four panels, the resource moves with it and ends with the
    // operand (rows behind the last panel read as zeros; columns behind the
    // last step are the next panel's, of outputs that do not exist).
    __device__ Feed(const PanelOperand& o, int32_t p0) {
      pitch = int64_t(o.steps) * 2048;
      data = o.data;
      first = p0;
      total = int64_t(o.rows16 / 16) * pitch;
      if constexpr (!T) {
        const int32_t n = o.rows16 / 16 - p0 < P ? o.rows16 / 16 - p0 : P;
        rsrc = panel_srd(data + p0 * pitch, uint32_t(n * pitch));
      }
    }
    __device__ __forceinline__ void prepare(int32_t s, int, int) {
      if constexpr (T) {
        const int64_t off = s * 4 * pitch + first * 512;
        const int64_t left = total - off;
        rsrc = panel_srd(data + off, uint32_t(left < 0 ? 0 : left < (int64_t(1) << 31) ? left : (int64_t(1) << 31)));
      }
    }
    __device__ __forceinline__ void put(int32_t s, uint32_t dst, int wave, int lane, int t) const {
      const int c = wave * LOADS + t;
      if constexpr (T) {
        constexpr int kChunks = P / 2;  // 32-column halves per panel
        const int from = (lane >> 4) * 256 + ((lane & 15) ^ ((lane >> 4 & 1) * 8)) * 16;
        panel_dma16(rsrc, dst + c * 1024, int32_t(c / kChunks * pitch) + c % kChunks * 1024 + from);
      } else {
        // panel c / 2, half c % 2
        panel_dma16(rsrc, dst + c * 1024, int32_t((c >> 1) * pitch) + s * 2048 + (c & 1) * 1024 + lane * 16);
      }
    }
  };

  // The same for A in tiles (PanelOperand).  A wavefront's four transfers are
  // two panels of one step in one tile (straight), or two steps of one panel
  // (transposed), each step in a tile column of its own.  The slots of 64
  // tiles at a time (of a tile row, or of the two tile columns) are held in
  // the lanes of a register.
  template <bool T, int P, int LOADS>
  struct TiledFeed {
    const PanelOperand& o;
    int32_t unit;         // first step (transposed) or first row (straight) of this wavefront
    int32_t first;        // tile column (straight) or row whose slot lane 0 holds
    int32_t slot0, slot1;
    int32_t now;          // tile column or row that the addresses are of
    const char *at0, *at1;
    srd4_t r0, r1;        // the prepared step's

    __device__ TiledFeed(const PanelOperand& op, int32_t p0, int wave)
        : o(op), first(-64), slot0(-1), slot1(-1), now(-1), at0(nullptr), at1(nullptr) {
      static_assert(LOADS == 4 && P == 16, "eight wavefronts, 256 rows or columns");
      unit = T ? p0 / 4 + (wave & 1) * 2 : (p0 + wave * 2) * 16;
    }
    // Address of tile (tn, tk) of the operand, or NULL.
    __device__ __forceinline__ const char* tile_at(int32_t tn, int32_t tk, int32_t slot) const {
      const bool dense = slot >= 0 && slot < o.n_dense && o.row0 + (int64_t(tn + 1) << o.log_b1) <= o.plain;
      if (!dense && (tn < o.spare0 || tn >= o.spare1)) return nullptr;
      const int64_t tile = dense ? slot : int64_t(tn - o.spare0) * o.tiles_k + tk;
      return (dense ? o.data : o.spare) + (tile << (o.log_b1 + o.log_b2 + 1));
    }
    // Straight: on entering a tile column, the address of the first step there
    // of this wavefront's first panel.
    __device__ __forceinline__ void enter_column(int32_t tk, int lane) {
      const int32_t tn = unit >> o.log_b1;
      const bool live = unit < o.rows16;  // a panel behind the operand reads as zeros
      if (tk < first || tk >= first + 64) {
        first = tk;
        const int64_t t = ((o.row0 >> o.log_b1) + tn) * o.tiles_k;
        slot0 = live && tk + lane < o.tiles_k ? o.tidx[t + tk + lane] : -1;
      }
      const int32_t slot = __builtin_amdgcn_readlane(slot0, tk - first);
      at0 = live ? tile_at(tn, tk, slot) : nullptr;
      if (at0) at0 += int64_t(unit & ((1 << o.log_b1) - 1)) << (o.log_b2 + 1);
    }
    // Transposed: on entering a tile row, the addresses of this wavefront's two
    // steps of the row's first panel.
    __device__ __forceinline__ void enter_row(int32_t tn, int lane) {
      const int shift = o.log_b2 - 6;
      if (tn < first || tn >= first + 64) {
        first = tn;
        const int32_t rows = (o.rows16 + (1 << o.log_b1) - 1) >> o.log_b1;
        const int64_t t = ((o.row0 >> o.log_b1) + tn + lane) * o.tiles_k;
        const bool in = tn + lane < rows;
        slot0 = in && unit < o.steps ? o.tidx[t + (unit >> shift)] : -1;
        slot1 = in && unit + 1 < o.steps ? o.tidx[t + ((unit + 1) >> shift)] : -1;
      }
      const int32_t mask = (1 << shift) - 1;
      const int32_t s0 = __builtin_amdgcn_readlane(slot0, tn - first), s1 = __builtin_amdgcn_readlane(slot1, tn - first);
      at0 = unit < o.steps ? tile_at(tn, unit >> shift, s0) : nullptr;
      at1 = unit + 1 < o.steps ? tile_at(tn, (unit + 1) >> shift, s1) : nullptr;
      if (at0) at0 += (unit & mask) * 2048;
      if (at1) at1 += ((unit + 1) & mask) * 2048;
    }
    __device__ __forceinline__ void prepare(int32_t s, int wave, int lane) {
      if constexpr (T) {
        const int32_t row = s * 64 + (wave >> 1) * 16, tn = row >> o.log_b1;
        if (tn != now) {
          now = tn;
          enter_row(tn, lane);
        }
        const bool live = row < o.rows16;
        const int32_t down = (row & ((1 << o.log_b1) - 1)) << (o.log_b2 + 1);
        r0 = panel_srd(at0 + down, live && at0 ? 2048 : 0);
        r1 = panel_srd(at1 + down, live && at1 ? 2048 : 0);
      } else {
        const int shift = o.log_b2 - 6;
        if (s >> shift != now) {
          now = s >> shift;
          enter_column(now, lane);
        }
        r0 = panel_srd(at0 + (s & ((1 << shift) - 1)) * 2048, at0 ? (32 << o.log_b2) + 2048 : 0);
      }
    }
    __device__ __forceinline__ void put(int32_t, uint32_t dst, int wave, int lane, int t) const {
      if constexpr (T) {
        const int from = (lane >> 4) * 256 + ((lane & 15) ^ ((lane >> 4 & 1) * 8)) * 16;
        panel_dma16(t < 2 ? r0 : r1, dst + (wave * 4 + t) * 1024, (t & 1) * 1024 + from);
      } else {
        // the tile's next panel is 32 b2 bytes on
        panel_dma16(r0, dst + (wave * 4 + t) * 1024, (t >> 1) * (32 << o.log_b2) + (t & 1) * 1024 + lane * 16);
      }
    }
  };

  // The same for A as codes read transposed: a step is four panels of 16 rows,
  // the tile's 256 columns two steps of each.  A wavefront transfers one.
  template <int P, int LOADS>
  struct CodesFeed {
    const PanelOperand& o;
    int32_t column;  // step of the panels
    srd4_t r;        // the prepared step's

    __device__ CodesFeed(const PanelOperand& op, int32_t p0, int wave) : o(op), column(p0 / 8 + (wave & 1)) {
      static_assert(LOADS == 2 && P == 16, "eight wavefronts, 256 columns");
    }
    __device__ __forceinline__ void prepare(int32_t s, int wave, int) {
      const int32_t panel = s * 4 + (wave >> 1);
      const bool live = panel * 16 < o.rows16 && column < o.steps;
      r = panel_srd(o.data + (live ? (int64_t(panel) * o.steps + column) * 2048 : 0), live ? 2048 : 0);
    }
    __device__ __forceinline__ void put(int32_t, uint32_t dst, int wave, int lane, int t) const {
      panel_dma16(r, dst + wave * 2048 + t * 1024, t * 1024 + lane * 16);
    }
  };

  // The two halves of panel p (of P) of a staged step.
  struct Halves {
    u32x4_t v[2];
  };
  template <bool T, int P>
  __device__ __forceinline__ static Halves read(const char* src, int p, int lane_off, int turn0, int turn1) {
    Halves r;
    if constexpr (T) {
      const char* c = src + (p >> 1) * 1024 + (p & 1) * 512;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const char* b = c + 2 * h * (P / 2) * 1024;
        const uint2 lo = __builtin_bit_cast(
            uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(const_cast<char*>(b + turn0))));
        const uint2 hi = __builtin_bit_cast(
            uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(const_cast<char*>(b + turn1))));
        r.v[h] = u32x4_t{lo.x, lo.y, hi.x, hi.y};
      }
    } else {
      const char* b = src + p * 2048 + lane_off;
      r.v[0] = *reinterpret_cast<const u32x4_t*>(b);
      r.v[1] = *reinterpret_cast<const u32x4_t*>(b + 1024);
    }
    return r;
  }

  // A's codes of column block p: the eight rows of each half step in the first
  // two words of its half.
  __device__ __forceinline__ static Halves read_codes(const char* src, int p, int off) {
    Halves r;
    const char* b = src + (p >> 3) * 2048 + ((p >> 2) & 1) * 1024 + (p & 3) * 256 + off;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint2 u = __builtin_bit_cast(
          uint2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2_t*)(const_cast<char*>(b + h * 8192))));
      r.v[h] = u32x4_t{u.x, u.y, 0, 0};
    }
    return r;
  }
  __device__ __forceinline__ static PanelRegs<KIND> widen_codes(const Halves& c, float scale) {
    PanelRegs<KIND> r;
    if constexpr (CODES) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (KIND == HYB_BF16) {
            r.v[h][2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.v[h][i], scale, false));
            r.v[h][2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.v[h][i], scale, true));
          } else {
            r.v[h][2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c.v[h][i], scale, false));
            r.v[h][2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c.v[h][i], scale, true));
          }
        }
    }
    return r;
  }

  // Lane offsets of the two transposing reads of a half: panel q/2 of the
  // half's two, rows 4 (q%2) + i (+ 8), columns 4 c.. of the block's 16.
  template <int P>
  __device__ __forceinline__ static int turn(int lane, int part) {
    const int q = lane >> 4, i = (lane & 15) >> 2, c = lane & 3;
    return (q >> 1) * (P / 2) * 1024 + (c >> 1) * 256 + (4 * (q & 1) + i + 8 * (part ^ (c >> 1))) * 16 + (c & 1) * 8;
  }

  // Sums of steps [s0, s1), s0 a multiple of four, of A panels pa.. and B
  // panels pb..; wavefront (wa, wb) ends with acc[i][j] of its panels
  // pa + wa kA + i, pb + wb kB + j (lane L: A rows 4 (L/16) + 0..3, B row L%16).
  __device__ static void run(const PanelOperand& A, const PanelOperand& B, int32_t pa, int32_t pb, int32_t s0,
                             int32_t s1, char* smem, f32x4_t (&acc)[kA][kB]) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wa = wave % WA, wb = wave / WA;
    auto fa = [&] {
      if constexpr (CODES)
        return CodesFeed<AP, kLoadsA>(A, pa, wave);
      else if constexpr (TILED)
        return TiledFeed<TA, AP, kLoadsA>(A, pa, wave);
      else
        return Feed<TA, AP, kLoadsA>(A, pa);
    }();
    Feed<TB, BP, kLoadsB> fb(B, pb);
    const uint32_t base = panel_lds_addr(smem);
    const int straight = lane * 16;
    const int ta0 = turn<AP>(lane, 0), ta1 = turn<AP>(lane, 1);
    const int tb0 = turn<BP>(lane, 0), tb1 = turn<BP>(lane, 1);
    [[maybe_unused]] const int codes_off =
        (lane >> 5) * 4096 + ((lane >> 4) & 1) * 128 + ((lane & 15) >> 1) * 16 + (lane & 1) * 8;
    [[maybe_unused]] const int codes_top = CODES && KIND == HYB_F16 ? int(*A.top) : 0;

    auto issue = [&](int32_t s, int stage) {
      const uint32_t dst = base + stage * kStage;
      fa.prepare(s, wave, lane);
#pragma unroll
      for (int t = 0; t < kLoadsA; ++t) fa.put(s, dst, wave, lane, t);
      fb.prepare(s, wave, lane);
#pragma unroll
      for (int t = 0; t < kLoadsB; ++t) fb.put(s, dst + kStageA, wave, lane, t);
      if constexpr (is_f8(KIND)) {
        // the scale words of steps s .. s+3: AP * 64 + BP * 64 bytes
        if ((s & 3) == 0) {
          const uint32_t sdst = base + STAGES * kStage + ((s >> 2) & 1) * kScaleStage;
          const int64_t word = int64_t(s >> 2);
          if (wave == 0) {
            const int32_t n = A.rows16 - pa * 16 < AP * 16 ? A.rows16 - pa * 16 : AP * 16;
            const srd4_t sa = panel_srd(A.scale + word * A.scale_pitch + pa * 16, uint32_t(n * 4));
            for (int c = 0; c * 1024 < AP * 64; ++c)
              if (lane * 16 + c * 1024 < AP * 64) panel_dma16(sa, sdst + c * 1024, lane * 16 + c * 1024);
          }
          if (wave == kWaves - 1) {
            const int32_t n = B.rows16 - pb * 16 < BP * 16 ? B.rows16 - pb * 16 : BP * 16;
            const srd4_t sb = panel_srd(B.scale + word * B.scale_pitch + pb * 16, uint32_t(n * 4));
            for (int c = 0; c * 1024 < BP * 64; ++c)
              if (lane * 16 + c * 1024 < BP * 64) panel_dma16(sb, sdst + AP * 64 + c * 1024, lane * 16 + c * 1024);
          }
        }
      }
    };

#pragma unroll
    for (int i = 0; i < kA; ++i)
#pragma unroll
      for (int j = 0; j < kB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    uint32_t sca[kA], scb[kB];
#pragma unroll
    for (int i = 0; i < kA; ++i) sca[i] = 0;
#pragma unroll
    for (int j = 0; j < kB; ++j) scb[j] = 0;

    // Scale of the codes of step s: this wavefront's columns lie in one step of
    // the panels, the step's 64 rows in one block.  The lanes hold the words of
    // 64 steps (a load for each step, waited for beside the LDS reads, cost a
    // trip to memory a step).
    [[maybe_unused]] float codes_scale = 1.f;
    [[maybe_unused]] uint32_t scale_words = 0;
    [[maybe_unused]] int32_t scale_first = s0 - 64;  // step of lane 0's word
    auto scale_word = [&](int32_t s) -> uint32_t {
      if constexpr (CODES) {
        const int32_t column = pa / 8 + wa * kA / 8, at = column < A.steps ? column : 0;
        if (s >= scale_first + 64) {
          scale_first = s;
          const int64_t row = int64_t(s + lane) * 64;
          scale_words = row < A.rows16 ? A.scale[int64_t(at >> 2) * A.scale_pitch + row] : 0;
        }
        return uint32_t(__builtin_amdgcn_readlane(int(scale_words), s - scale_first)) >> (8 * (at & 3));
      }
      return 0;
    };
    auto set_scale = [&](uint32_t word) {
      int byte8 = int(word & 0xFFu);
      if constexpr (KIND == HYB_F16) {
        byte8 += 133 - codes_top;
        byte8 = byte8 < 1 ? 1 : byte8;
      }
      codes_scale = __builtin_bit_cast(float, uint32_t(byte8) << 23);
    };

    // Multiplies the staged step s and, once its first reads are under way,
    // starts the transfers of step s + STAGES - 1: at once, or (kSpread) two
    // between the products of each A panel, where a transfer waits for the
    // address unit without holding up the products.  That serves the product
    // over codes, whose vector unit is busy widening (1000 tokens x 152064 x
    // 5120 with dX 4145 -> 4045 us); the 16-bit ones lose by it, their
    // transfers arriving late (dX piece 832 -> 868 us, dW 869 -> 926, logits
    // even).  The reads of A panel i + 1 are issued ahead of panel i's
    // products, so that an LDS round trip hides behind them (the scheduling
    // barriers keep the compiler from moving them back).
    constexpr bool kSpread = CODES && STAGES == 2 && kB % 2 == 0 && 2 * kA >= kLoadsA + kLoadsB;
    auto compute = [&](int32_t s, int stage, auto byte, bool more) {
      constexpr int kByte = decltype(byte)::value;
      const char* src = smem + stage * kStage;
      const char* srcb = src + kStageA;
      if constexpr (is_f8(KIND)) {
        if (kByte == 0) {
          const char* sc = smem + STAGES * kStage + ((s >> 2) & 1) * kScaleStage + (lane & 15) * 4;
#pragma unroll
          for (int i = 0; i < kA; ++i) sca[i] = *reinterpret_cast<const uint32_t*>(sc + (wa * kA + i) * 64);
#pragma unroll
          for (int j = 0; j < kB; ++j) scb[j] = *reinterpret_cast<const uint32_t*>(sc + (AP + wb * kB + j) * 64);
        }
      }
      auto read_a = [&](int i) {
        if constexpr (CODES) return read_codes(src, wa * kA + i, codes_off);
        else return read<TA, AP>(src, wa * kA + i, straight, ta0, ta1);
      };
      // Rows behind the last that counts: their codes, whatever they are, zero.
      auto mask_codes = [&](Halves& c) {
        const int64_t left = A.plain - int64_t(s) * 64;
        if (left >= 64) return;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int32_t keep = int32_t(left) - 32 * h - 16 * (lane >> 5) - 8 * ((lane >> 4) & 1);
          const uint64_t m = keep <= 0 ? 0 : keep >= 8 ? ~uint64_t(0) : (uint64_t(1) << (8 * keep)) - 1;
          c.v[h][0] &= uint32_t(m);
          c.v[h][1] &= uint32_t(m >> 32);
        }
      };
      Halves a = read_a(0);
      Halves braw[kB];
#pragma unroll
      for (int j = 0; j < kB; ++j) braw[j] = read<TB, BP>(srcb, wb * kB + j, straight, tb0, tb1);
      [[maybe_unused]] const uint32_t next_dst = base + ((stage + STAGES - 1) % STAGES) * kStage;
      if (more) {
        if constexpr (kSpread) {
          fa.prepare(s + 1, wave, lane);
          fb.prepare(s + 1, wave, lane);
        } else {
          issue(s + STAGES - 1, (stage + STAGES - 1) % STAGES);
        }
      }
      [[maybe_unused]] uint32_t next_word = 0;
      if constexpr (CODES)
        if (s + 1 < s1) next_word = scale_word(s + 1);
      PanelRegs<KIND> b[kB];
#pragma unroll
      for (int j = 0; j < kB; ++j) b[j] = panel_regs<KIND, kByte>(braw[j].v[0], braw[j].v[1], scb[j]);
#pragma unroll
      for (int i = 0; i < kA; ++i) {
        const Halves was = a;
        if (i + 1 < kA) a = read_a(i + 1);
        PanelRegs<KIND> now;
        if constexpr (CODES) {
          Halves c = was;
          mask_codes(c);
          now = widen_codes(c, codes_scale);
        } else {
          now = panel_regs<KIND, kByte>(was.v[0], was.v[1], sca[i]);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < kB; ++j) {
          acc[i][j] = panel_mfma<KIND, kByte>(now, b[j], acc[i][j], sca[i], scb[j]);
          if constexpr (kSpread) {
            const int t = 2 * i + j / (kB / 2);
            if (j % (kB / 2) == kB / 2 - 1 && t < kLoadsA + kLoadsB) {
              __builtin_amdgcn_sched_barrier(0);
              if (more) {
                if (t < kLoadsA)
                  fa.put(s + 1, next_dst, wave, lane, t);
                else
                  fb.put(s + 1, next_dst + kStageA, wave, lane, t - kLoadsA);
              }
              __builtin_amdgcn_sched_barrier(0);
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (CODES) set_scale(next_word);
    };

    // A step waits for its own transfers (those of the STAGES - 2 steps after it
    // may be under way; the few scale transfers only make that wait
    // stricter) and meets the other wavefronts, whose reads of the stage
    // that is filled next are then done too.  Unrolled by four so that stage
    // and scale byte are immediates.
    if (s0 >= s1) return;
    if constexpr (CODES) set_scale(scale_word(s0));
#pragma unroll
    for (int t = 0; t < STAGES - 1; ++t)
      if (s0 + t < s1) issue(s0 + t, t);
    for (int32_t q = s0; q < s1; q += 4) {
      auto one = [&](auto byte) {
        constexpr int kByte = decltype(byte)::value;
        const int32_t s = q + kByte;
        if (s >= s1) return;
        if (STAGES > 2 && s + STAGES - 2 < s1)
          panel_wait<(STAGES - 2) * (kLoadsA + kLoadsB)>();
        else
          panel_wait<0>();
        __syncthreads();
        compute(s, kByte % STAGES, byte, s + STAGES - 1 < s1);
      };
      one(std::integral_constant<int, 0>());
      one(std::integral_constant<int, 1>());
      one(std::integral_constant<int, 2>());
      one(std::integral_constant<int, 3>());
    }
  }
};

}  // namespace
}  // namespace hyb

#endif  // HYB_PANEL_H_
