// Linear attention with a decay for each head on gfx950: the chunked forward and backward.
//
// Per head, S_t = e^{g_t} S_{t-1} + k_t v_t^T and o_t = scale S_t^T q_t.  Within a 64-token chunk
// with G the cumulative sum of g and S the state at the chunk's start,
//   o_t = scale (e^{G_t} S^T q_t + sum_{i <= t} e^{G_t - G_i} (q_t . k_i) v_i)
//   S  <- e^{G_C} S + sum_i e^{G_C - G_i} k_i v_i^T.
// The gradients are the same recurrence with other rows: dq_t = scale S_t do_t reads the state
// built from (v, k); with dS the gradient of the state, dS_{t-1} = e^{g_t} dS_t-like recurrences
// run backward in time on (q, do), and dv_t = dS_t^T k_t, dk_t = dS_t v_t.  So one kernel does all
// of them (LinPass).  Nothing couples the columns of the state, and sequences are split into units
// of L chunks exactly: a unit's own sum from zero (kLinSum*), the sums joined along the sequence
// (lin_scan_kernel), the unit run from its true start.  The backward's passes of one stage are one
// launch (kGroupSums, kGroupGrads).
//
// Work of one workgroup (4 waves, 8 where it has a CU to itself): one (unit, head).  Wave w owns
// D / 4 (or D / 8) columns of the state, all D rows of them, in MFMA accumulators: in that layout
// (lane n + 16 (m / 4), item m % 4) two stacked 16-row tiles are, as they stand, the operand of a
// 16x16x32 product over the rows, in the row order {4 gq + j, 16 + 4 gq + j}.  All row operands are
// read in that order, so the state never passes through LDS.  The masked 64 x 64 products P are
// formed once per workgroup, ten 16 x 16 tiles over four waves, and pass through LDS in operand
// order.  Output tiles are formed transposed (columns by items), so a lane stores 16 consecutive
// bytes of a row.
//
// Rounding: inputs are bf16, sums and states fp32.  Products take bf16 operands; what is not an
// input is split into a sum of bf16 terms: two terms (2^-17) where the result is rounded to bf16
// in the end, three (2^-25) where it is kept in fp32 (final states, state gradients, dg's parts).
// One term of the state is not enough for o and dv: its rounding goes with the size of the terms
// q_i S_ij, not of their sum, which is far smaller where keys share a direction that the query does
// not (keys of weight 4 in one direction against unit noise: 8.5e-2 of o, two terms 1.7e-3).
// fp32 inputs use the fp32 MFMA throughout.
//
// What bounds it (one MI355X, d = 128, bf16).  200K tokens x 16 heads forward: 0.87 ms for 3.36 GB,
// 3.9 TB/s; the kernel's loads and stores alone take 0.73 ms there, its products on rows that stay
// in the caches 0.72 ms.  65K tokens x 8 heads backward: sums 159, scan 21, gradients 572, dg 17 us;
// the gradients alone move 2.05 GB (3.6 TB/s), and on rows that stay in the caches they still take
// 476 us: per SIMD the matrix unit is busy 32 % of the time, vector issue 31 % (without MFMA), LDS
// 32 %, and two waves per SIMD (256 registers each) overlap them only in part.  Fewer vector
// instructions (decays folded into the state's share: 64 of some 900 per chunk) and passes of one
// unit placed side by side on one XCD (677 against 661 us) did not shorten it.
//
// Decays: G in units of log2, accumulated as a pair of floats (hi + lo), and only differences of G
// are exponentiated, so no factor overflows and far tokens keep their precision.  Log decays below
// kMinLog2 have no fp32 value above zero and are taken as kMinLog2: -inf empties the state.
#include <algorithm>
#include <atomic>

#include "gdn_device.h"
#include "gdn_internal.h"
#include "gdn_linattn.h"
#include "gdn_unit.h"

namespace gdn {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr float kMinLog2 = -512.f;
constexpr float kNoDecay = -150.f;  // 2^-150 rounds to zero in fp32
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eLo = 1.925963033500e-8f;  // log2(e) - kLog2e

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Sums of floats kept as hi + lo.
struct F2 {
  float hi, lo;
};
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  const float s = a.hi + b.hi, bb = s - a.hi;
  const float e = (a.hi - (s - bb)) + (b.hi - bb);
  return F2{s, a.lo + b.lo + e};
}
template <int CTRL, int MASK>
__device__ __forceinline__ F2 scan_step(F2 x) {
  return add2(x, F2{dpp_moved<CTRL, MASK>(x.hi), dpp_moved<CTRL, MASK>(x.lo)});
}
// Inclusive sum over the wave's 64 lanes.
__device__ __forceinline__ F2 wave_scan2(F2 x) {
  x = scan_step<0x111, 0xf>(x);
  x = scan_step<0x112, 0xf>(x);
  x = scan_step<0x114, 0xf>(x);
  x = scan_step<0x118, 0xf>(x);
  x = scan_step<0x142, 0xa>(x);
  x = scan_step<0x143, 0xc>(x);
  return x;
}
// A natural-log decay in log2 units.
__device__ __forceinline__ F2 log2_decay(float g) {
  const float hi = g * kLog2e;
  if (hi < kMinLog2) return F2{kMinLog2, 0.f};  // NaN passes on
  return F2{hi, __builtin_fmaf(g, kLog2e, -hi) + g * kLog2eLo};
}

// The operands of a product over 32 indices, in the order {4 gq + j, 16 + 4 gq + j} (j < 4), and
// the product itself, for both input types.
template <class E>
struct Op;
// bf16 tiles in LDS.  Tiles of which rows and columns are read (y, z): rows of D + 16 elements, 8
// (mod 64) banks apart, with the 16-byte units exchanged in pairs in every other group of eight
// rows, so that the eight rows of a transposing read's half wave lie on different banks.  Tiles of
// which only rows are read (x, w): rows of D + 4 elements, whose 16 rows' 8-byte reads of one cycle
// fill the 32 banks.
template <>
struct Op<bf16> {
  typedef bf16x8 Frag;
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  static constexpr int kPadYZ = 16, kPadXW = 4;
  // where column `col` of row `row` of y or z is within the row (col a multiple of 4)
  static __device__ __forceinline__ int place(int row, int col) { return col ^ (row & 8); }
  static __device__ __forceinline__ void put_xw(bf16 *p, u32x4 x) {  // 8-byte aligned
    *reinterpret_cast<u32x2 *>(p) = __builtin_shufflevector(x, x, 0, 1);
    *reinterpret_cast<u32x2 *>(p + 4) = __builtin_shufflevector(x, x, 2, 3);
  }
  static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) { return mma_bf16(a, b, c); }
  // a row, from its element at index 4 gq on (a multiple of 32 further: the next products')
  static __device__ __forceinline__ Frag row(const bf16 *p) {
    return cat8(lds_bf16x4(p), lds_bf16x4(p + 16));
  }
  // a column: rows row0 + (order) of the tile's column that the lane's offset `at` is for
  // (colq: the first of the four columns that the lane addresses in the transposing read)
  static __device__ __forceinline__ int column_base(int colq, int, int c, int gq, int ld) {
    const int r = 4 * gq + (c >> 2);
    return r * ld + place(r, colq);
  }
  template <int LD>
  static __device__ __forceinline__ Frag column(const bf16 *tile, int at) {
    return cat8(lds_tr16(tile + at), lds_tr16(tile + at + 16 * LD));
  }
  static __device__ __forceinline__ Frag round(f32x4 a, f32x4 b) { return to_bf16x8(a, b); }
  // a, b less what round() made of them: x - hi is one dot product with (-1, 0) or (0, -1).  The
  // pairs are kept in registers: as an inline constant the compiler writes (-1, 0) as the fp32
  // -1.0, which is the other pair.
  static __device__ __forceinline__ void residual(Frag f, f32x4 &a, f32x4 &b) {
    unsigned u0 = 0x0000bf80u, u1 = 0xbf800000u;
    asm("" : "+s"(u0), "+s"(u1));
    const bf16x2 e0 = __builtin_bit_cast(bf16x2, u0), e1 = __builtin_bit_cast(bf16x2, u1);
    const bf16x2 f0 = {f[0], f[1]}, f1 = {f[2], f[3]}, f2 = {f[4], f[5]}, f3 = {f[6], f[7]};
    a = f32x4{__builtin_amdgcn_fdot2_f32_bf16(f0, e0, a[0], false),
              __builtin_amdgcn_fdot2_f32_bf16(f0, e1, a[1], false),
              __builtin_amdgcn_fdot2_f32_bf16(f1, e0, a[2], false),
              __builtin_amdgcn_fdot2_f32_bf16(f1, e1, a[3], false)};
    b = f32x4{__builtin_amdgcn_fdot2_f32_bf16(f2, e0, b[0], false),
              __builtin_amdgcn_fdot2_f32_bf16(f2, e1, b[1], false),
              __builtin_amdgcn_fdot2_f32_bf16(f3, e0, b[2], false),
              __builtin_amdgcn_fdot2_f32_bf16(f3, e1, b[3], false)};
  }
  // two stored tiles side by side
  static __device__ __forceinline__ Frag pair(const bf16 *p, int next) {
    return cat8(lds_bf16x4(p), lds_bf16x4(p + next));
  }
  static __device__ __forceinline__ f32x4 lo_part(Frag f) {
    return f32x4{(float)f[0], (float)f[1], (float)f[2], (float)f[3]};
  }
  static __device__ __forceinline__ f32x4 hi_part(Frag f) {
    return f32x4{(float)f[4], (float)f[5], (float)f[6], (float)f[7]};
  }
};
struct F32x8 {
  f32x4 a, b;
};
template <>
struct Op<float> {
  typedef F32x8 Frag;
  static constexpr int kPadYZ = 4, kPadXW = 4;
  static __device__ __forceinline__ int place(int, int col) { return col; }
  static __device__ __forceinline__ void put_xw(float *p, u32x4 x) { *reinterpret_cast<u32x4 *>(p) = x; }
  static __device__ __forceinline__ f32x4 mma(Frag x, Frag y, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = mma_f32(x.a[j], y.a[j], c);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = mma_f32(x.b[j], y.b[j], c);
    return c;
  }
  static __device__ __forceinline__ Frag row(const float *p) {
    return F32x8{lds_f32x4(p), lds_f32x4(p + 16)};
  }
  static __device__ __forceinline__ int column_base(int, int col, int, int gq, int ld) {
    return 4 * gq * ld + col;
  }
  template <int LD>
  static __device__ __forceinline__ Frag column(const float *tile, int at) {
    const float *p = tile + at;
    F32x8 f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f.a[j] = p[j * LD];
      f.b[j] = p[(16 + j) * LD];
    }
    return f;
  }
  static __device__ __forceinline__ Frag round(f32x4 a, f32x4 b) { return F32x8{a, b}; }
  static __device__ __forceinline__ void residual(Frag, f32x4 &, f32x4 &) {}
  static __device__ __forceinline__ Frag pair(const float *p, int next) {
    return F32x8{lds_f32x4(p), lds_f32x4(p + next)};
  }
  static __device__ __forceinline__ f32x4 lo_part(Frag f) { return f.a; }
  static __device__ __forceinline__ f32x4 hi_part(Frag f) { return f.b; }
};

template <class E>
__device__ __forceinline__ void store4(E *p, f32x4 x);
template <>
__device__ __forceinline__ void store4<float>(float *p, f32x4 x) {
  *reinterpret_cast<f32x4 *>(p) = x;
}
template <>
__device__ __forceinline__ void store4<bf16>(bf16 *p, f32x4 x) {
  *reinterpret_cast<bf16x4 *>(p) = to_bf16x4(x);
}
__device__ __forceinline__ f32x4 load4(const bf16 *p) {
  const bf16x4 x = lds_bf16x4(p);
  return f32x4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
}
__device__ __forceinline__ f32x4 load4(const float *p) { return lds_f32x4(p); }

// x where d <= 0, else zero (whatever x is): a select would cost a compare and, at three times a
// vector operation's rate, the select itself.
__device__ __forceinline__ float kept(float x, int d) {
  return __int_as_float(__float_as_int(x) & ((d - 1) >> 31));
}

// Sums over the wave's four rows of 16 lanes, of two values at once: the halves of a and b are
// exchanged (lanes 32 and up of a with the others of b), so one addition adds both over the halves,
// a's in lanes 0 to 31; the same again by rows.
__device__ __forceinline__ float halves_sum(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float rows_sum(float a, float b) {  // rows 0, 2: a's pairs of rows; 1, 3: b's
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <int PASS>
struct PassTraits {
  static constexpr bool kSum = PASS == kLinSumFwd || PASS == kLinSumRev;
  static constexpr bool kRev = PASS == kLinDv || PASS == kLinDk || PASS == kLinSumRev;
  static constexpr bool kTransposed = PASS == kLinDq || PASS == kLinDk;  // state rows = v, do
  static constexpr bool kDots = PASS == kLinDq || PASS == kLinDk;        // parts of dg
  static constexpr bool kGrad = PASS != kLinFwd && PASS != kLinSumFwd;
  static constexpr int kTiles = kSum ? 2 : (kDots ? 4 : 3);
};

// The 64 x 64 products P in LDS, by 16 x 16 tiles (16 rows of x, 16 of y) in operand order: the
// tiles that a row of tiles needs (two at a time; a masked partner is stored as zeros).
template <bool REV>
__device__ __forceinline__ int p_slot(int xt, int yt) {
  if (REV) return (xt == 0 ? 0 : xt == 1 ? 4 : xt == 2 ? 8 : 10) + yt - (xt & 2);
  return (xt == 0 ? 0 : xt == 1 ? 2 : xt == 2 ? 4 : 8) + yt;
}
constexpr int kPSlots = 12;
template <class E>
constexpr int p_terms() {
  return sizeof(E) == 2 ? 2 : 1;
}
template <class E>
constexpr size_t p_bytes() {
  return (size_t)kPSlots * 64 * 4 * sizeof(E) * p_terms<E>();
}

template <class E, int D, int PASS>
constexpr size_t pass_lds_bytes() {
  typedef PassTraits<PASS> PT;
  const int elems = 2 * 64 * (D + Op<E>::kPadYZ) + (PT::kTiles - 2) * 64 * (D + Op<E>::kPadXW);
  return elems * sizeof(E) + (PT::kSum || PT::kDots ? 0 : p_bytes<E>());
}

}  // namespace

template <int WAVES>
struct PassShared {
  // the chunk's decays, by its parity: G (log2, hi + lo) and the factors of x's and y's rows
  __attribute__((aligned(16))) float s_hi[2][64], s_lo[2][64], s_x[2][64], s_yf[2][64];
  // dg's parts, by the chunk's parity; the pairs' row sums (in the block on the diagonal, off it) and
  // the columns' sums over each wave's tiles
  __attribute__((aligned(16))) float csum[2][4][32];
  float dots[2][WAVES][64], rsum[2][2][64];
  float s_decay[2];
  int unit[4];
};

// SETS: chunks whose rows are on their way in registers (sums: one or two; two set launch bounds that
// hold two workgroups per CU, one three).
template <class E, int D, int PASS, int WAVES, int SETS>
__device__ __forceinline__ void lin_pass(const LinArgs &a, char *smem, PassShared<WAVES> &sh) {
  typedef Op<E> X;
  typedef typename X::Frag Frag;
  typedef PassTraits<PASS> PT;
  constexpr int NT = D / (16 * WAVES);  // 16-column tiles of the state per wave
  constexpr int LDY = D + X::kPadYZ, LDX = D + X::kPadXW;
  constexpr int MT = D / 16;      // 16-row tiles of the state
  constexpr int KS = D / 32;      // products over a row
  constexpr int EPU = 16 / (int)sizeof(E);
  constexpr int UPR = D / EPU;            // 16-byte units per row
  constexpr int UPT = UPR / WAVES;        // ... per thread and tile
  // terms of the split operands (see the file's head)
  constexpr bool kB = sizeof(E) == 2;
  constexpr int kStateTerms = !kB ? 1 : (PT::kDots ? 3 : 2);
  constexpr int kPTerms = p_terms<E>();
  constexpr int kDecayWave = WAVES - 1;

  E *const ty = reinterpret_cast<E *>(smem);   // tiles of 64 rows
  E *const tz = ty + 64 * LDY;
  E *const tx = tz + 64 * LDY;
  E *const tw = tx + 64 * LDX;
  // P: behind the tiles, or (four tiles) over x, which is dead by then
  E *const tp = PT::kDots ? tx : tx + 64 * LDX;
  auto &s_hi = sh.s_hi, &s_lo = sh.s_lo, &s_x = sh.s_x, &s_yf = sh.s_yf;
  auto &dots = sh.dots;
  auto &rsum = sh.rsum;
  auto &csum = sh.csum;
  auto &s_decay = sh.s_decay;
  auto &sh_unit = sh.unit;

  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, gq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int unit = a.longest_first ? blockIdx.y : blockIdx.x;
  const int h = a.longest_first ? blockIdx.x : blockIdx.y;
  const int hk = __builtin_amdgcn_readfirstlane(h / (a.H / a.HK));

  if (w == 0) {
    Unit un{};
    const bool ok = find_unit(a.cu, a.N, a.T, a.L, unit, false, lane, un, a.longest_first != 0);
    if (lane == 0) {
      sh_unit[0] = ok ? un.seq : -1;
      sh_unit[1] = un.c0;
      sh_unit[2] = un.c1;
    }
  }
  __syncthreads();
  const int seq = __builtin_amdgcn_readfirstlane(sh_unit[0]);
  const int c0 = __builtin_amdgcn_readfirstlane(sh_unit[1]);
  const int c1 = __builtin_amdgcn_readfirstlane(sh_unit[2]);
  if (seq < 0) return;
  // uniform, and known to be: the rows' addresses are made of scalars
  const int64_t t_beg = __builtin_amdgcn_readfirstlane(a.cu[seq]);
  const int64_t t_end = __builtin_amdgcn_readfirstlane(a.cu[seq + 1]);
  if (t_beg < 0 || t_end < t_beg || t_end > a.T) return;
  const int nch = (int)((t_end - t_beg + kChunk - 1) / kChunk);
  const bool first = c0 == 0, last = c1 >= nch;
  const bool edge_in = PT::kRev ? last : first;    // the pass starts at the sequence's edge
  const bool edge_out = PT::kRev ? first : last;   // ... ends there
  // a whole sequence's index is the sequence, whatever the order they are taken in
  const int64_t uh = (int64_t)(a.L > 0 ? unit : seq) * a.H + h;
  if (PT::kSum) {
    if (PASS == kLinSumFwd && first && h == 0 && tid == 0) a.seq_unit[seq] = unit;
    if (edge_out) return;  // no unit follows
  }

  // the rows of this pass, and which of them are key heads'
  constexpr bool kXk = PASS == kLinFwd || PASS == kLinDv, kYk = PT::kSum || kXk, kZk = PT::kDots;
  const void *px = nullptr, *py, *pz, *pw = nullptr;
  if (PASS == kLinFwd) {
    px = a.q, py = a.k, pz = a.v;
  } else if (PASS == kLinDq) {
    px = a.dout, py = a.v, pz = a.k, pw = a.q;
  } else if (PASS == kLinDv) {
    px = a.k, py = a.q, pz = a.dout;
  } else if (PASS == kLinDk) {
    px = a.v, py = a.dout, pz = a.q, pw = a.k;
  } else if (PASS == kLinSumFwd) {
    py = a.k, pz = a.v;
  } else {
    py = a.q, pz = a.dout;
  }
  const float s_out = PASS == kLinFwd || PASS == kLinDq ? a.scale : 1.f;  // of the state's share
  const float s_p = a.scale;                                              // of P
  const float s_y = PT::kRev ? a.scale : 1.f;                             // of what enters the state

  // this wave's columns of the state: tile t's column of lane c, and the first column that the
  // lane addresses in a transposing read; in an output tile the lane has columns out_col + 4 t ..
  const int col = NT == 2 ? 32 * w + 8 * (c >> 2) + (c & 3) : 16 * w + c;  // (tile 1: 4 further)
  const int z_at = X::column_base(NT == 2 ? 32 * w + 8 * (c & 3) : 16 * w + 4 * (c & 3), col, c, gq, LDY);
  const int y_at = X::column_base(4 * (c & 3), c, c, gq, LDY);
  const int out_col = NT == 2 ? 32 * w + 8 * gq : 16 * w + 4 * gq;
  const int row_y = X::place(c, 4 * gq);    // a row operand's first element in y or z (rows 16 i + c)

  void *const out = PASS == kLinFwd ? a.o : PASS == kLinDq ? a.dq : PASS == kLinDk ? a.dk : a.dv;
  float *const final_state = PASS == kLinFwd ? a.ht : PASS == kLinDv ? a.dh0 : nullptr;
  const bool f32_out = PT::kDots && a.grad_f32;   // dq, dk of grouped heads: fp32 per value head
  const bool per_k = PT::kDots && !f32_out;
  const int out_heads = per_k ? a.HK : a.H, out_head = per_k ? hk : h;

  f32x4 S[MT][NT];
  const float *src = nullptr;
  if (!PT::kSum) {
    if (edge_in)
      src = PT::kRev ? (a.dht ? a.dht + ((int64_t)seq * a.H + h) * D * D : nullptr)
                     : (a.h0 ? a.h0 + seq * a.h0_stride + (int64_t)h * D * D : nullptr);
    else
      src = (PT::kRev ? a.unit_r : a.unit_s) + uh * D * D;
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      S[m][t] = zero4();
      if (src) {
        const int r = 16 * m + 4 * gq;
        if (PT::kTransposed) {
          S[m][t] = *reinterpret_cast<const f32x4 *>(src + (col + 4 * t) * D + r);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) S[m][t][j] = src[(r + j) * D + col + 4 * t];
        }
      }
    }

  // rows that are on their way, and their log decays (one wave): the next chunk's, or the next two
  // chunks' (the sums' rounds are short against a load's latency)
  constexpr int kSets = SETS;
  struct Rows {
    u32x4 y[UPT], z[UPT], x[UPT], w[UPT];
    float g;
  };
  Rows set[kSets];
  // Rows are read and written through buffer resources of the chunk's rows: the base is scalar, a
  // lane holds one 32-bit offset per row stride, and rows past the sequence's end are out of the
  // buffer's range, so they read as zeros and are not written.
  const int r0 = tid / UPR, o0 = tid % UPR * EPU;
  constexpr int kRows = 64 * WAVES / UPR;  // rows per round
  const auto rows_of = [&](const void *base, int64_t t0, int heads, int head, int n, int size) {
    const char *p = static_cast<const char *>(base) + (t0 * heads + head) * D * size;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), (short)0,
                                             ((n - 1) * heads + 1) * D * size, 0x00020000);
  };
  const auto load_rows = [&](u32x4(&to)[UPT], const void *base, int64_t t0, bool of_k, int n) {
    const int heads = of_k ? a.HK : a.H;
    const auto rsrc = rows_of(base, t0, heads, of_k ? hk : h, n, sizeof(E));
    int mine = tid;
    asm("" : "+v"(mine));  // the lane's offset in the first round's rows: made here, not kept
    const int at = (mine / UPR * heads * D + mine % UPR * EPU) * (int)sizeof(E);
#pragma unroll
    for (int u = 0; u < UPT; ++u)
      to[u] = __builtin_amdgcn_raw_buffer_load_b128(
          rsrc, at + kRows * u * heads * D * (int)sizeof(E), 0, 0);
  };
  const auto fetch = [&](Rows &to, int ch) {
    const int64_t t0 = t_beg + (int64_t)ch * kChunk;
    const int n = (int)(t_end - t0 < kChunk ? t_end - t0 : kChunk);
    load_rows(to.y, py, t0, kYk, n);
    load_rows(to.z, pz, t0, kZk, n);
    if (!PT::kSum) load_rows(to.x, px, t0, kXk, n);
    if (PT::kDots) load_rows(to.w, pw, t0, true, n);
    if (w == kDecayWave) to.g = lane < n ? a.g[a.g_head ? h : (t0 + lane) * a.H + h] : 0.f;
  };
  // the decays of the chunk that was fetched (one wave)
  F2 total{0.f, 0.f};  // the unit's whole log decay
  const auto make_decays = [&](float g, int par) {
    const F2 G = wave_scan2(log2_decay(g));
    const F2 GC = F2{__shfl(G.hi, 63, 64), __shfl(G.lo, 63, 64)};
    const float from_start = exp2_fast(G.hi + G.lo);
    const float to_end = exp2_fast((GC.hi - G.hi) + (GC.lo - G.lo));
    s_x[par][lane] = s_out * (PT::kRev ? to_end : from_start);
    s_yf[par][lane] = PT::kRev ? s_y * from_start : to_end;
    if (lane == 0) s_decay[par] = exp2_fast(GC.hi + GC.lo);
    if (PT::kSum) {
      total = add2(total, GC);
    } else {
      s_hi[par][lane] = G.hi;
      s_lo[par][lane] = G.lo;
    }
  };
  // dg's parts of the chunk before (every wave's share is in LDS)
  const auto flush_dots = [&](int ch, int par) {
    if (!PT::kDots || w != kDecayWave) return;
    const int64_t t = t_beg + (int64_t)ch * kChunk + lane;
    float *const to = PASS == kLinDq ? a.dg_q : a.dg_k;
    float d = dots[par][0][lane];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) d += dots[par][i][lane];
    if (t < t_end) to[(int64_t)h * a.T + t] = d;
    if (PASS == kLinDq) {
      // sum over the pairs s >= t > i = sum_{s >= t} (row sum - column sum); rows from the end.  The
      // first 32 rows have pairs in their own block only, the others' columns too.
      F2 x = F2{rsum[par][0][lane], 0.f};
      if (lane < 32) {
        x = add2(x, F2{-csum[par][0][lane], 0.f});
        x = add2(x, F2{-csum[par][1][lane], 0.f});
        x = add2(x, F2{-csum[par][3][lane], 0.f});
      } else {
        x = add2(x, F2{rsum[par][1][lane], 0.f});
        x = add2(x, F2{-csum[par][2][lane - 32], 0.f});
      }
      const F2 up = wave_scan2(x);
      const float th = __shfl(up.hi, 63, 64), tl = __shfl(up.lo, 63, 64);
      const F2 rest = add2(add2(F2{th, tl}, F2{-up.hi, -up.lo}), x);
      if (t < t_end) a.dg_pairs[(int64_t)h * a.T + t] = rest.hi + rest.lo;
    }
  };

  const int step = PT::kRev ? -1 : 1;
  int ch = PT::kRev ? c1 - 1 : c0;
  const int nsteps = c1 - c0;
  // terms of the state update: three where the state is written out or feeds dg
  const bool precise = kB && (PT::kSum || PT::kDots || (edge_out && final_state != nullptr));
  if (nsteps > 0) {
    fetch(set[0], ch);
    if (kSets > 1 && nsteps > 1) fetch(set[kSets - 1], ch + step);
    if (w == kDecayWave) make_decays(set[0].g, 0);
  }
  // one chunk, whose rows are in `in`; `next` holds the next chunk's
  const auto round = [&](int it, Rows &in, Rows &next) {
    const int64_t t0 = t_beg + (int64_t)ch * kChunk;
    const int par = it & 1;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      const int row = r0 + kRows * u, oy = row * LDY + X::place(row, o0), ox = row * LDX + o0;
      *reinterpret_cast<u32x4 *>(ty + oy) = in.y[u];
      *reinterpret_cast<u32x4 *>(tz + oy) = in.z[u];
      if (!PT::kSum) X::put_xw(tx + ox, in.x[u]);
      if (PT::kDots) X::put_xw(tw + ox, in.w[u]);
    }
    __syncthreads();
    const float *const g_hi = s_hi[par], *const g_lo = s_lo[par], *const f_x = s_x[par], *const f_y = s_yf[par];
    if (it > 0) flush_dots(ch - step, par ^ 1);
    // the next chunk's loads: at once, or (four tiles) once the first half's registers are free
    if (!PT::kDots && it + kSets < nsteps) fetch(in, ch + kSets * step);

    Frag zf[2][NT];  // z's columns of this wave: rows 32 kb + (order)
    const auto read_z = [&]() {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int t = 0; t < NT; ++t) zf[kb][t] = X::template column<LDY>(tz + 32 * kb * LDY + 4 * t, z_at);
    };
    if constexpr (PT::kSum && kSets > 1) read_z();

    f32x4 o[4][NT];  // the output by 16-row tiles
    if constexpr (!PT::kSum) {
      // the pairs within the chunk: P's ten 16 x 16 tiles, two or three per wave.  Waves 0 and 2: the
      // 32 x 32 blocks on the diagonal (two tiles masked within, one whole, one that is zero); waves
      // 1 and 3: 16 rows of x each of the block off it.
      // (Of eight waves, 4 to 7 go on to the state's share.)
      const bool forms_p = WAVES == 4 || w < 4, diag = (w & 1) == 0;
      const int xb = diag ? 16 * w : PT::kRev ? 16 * (w >> 1) : 32 + 16 * (w >> 1);  // first row of x
      const int yb = diag ? 16 * w : PT::kRev ? 32 : 0;                             // ... of y
      f32x4 p[3];  // on the diagonal: (0, 0), the whole one, (1, 1); off it: y's two tiles
      float r_sum[2] = {0.f, 0.f};
      const E *const xrow = tx + (xb + c) * LDX + 4 * gq, *const yrow = ty + (yb + c) * LDY + row_y;
      const E *const wrow = tw + (xb + c) * LDX + 4 * gq, *const zrow = tz + (yb + c) * LDY + row_y;
      const auto tiles = [&](const E *xr, const E *yr, f32x4(&acc)[3]) {
        acc[0] = acc[1] = acc[2] = zero4();
        if (diag) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const Frag x_0 = X::row(xr + 32 * ks), x_1 = X::row(xr + 16 * LDX + 32 * ks);
            const Frag y_0 = X::row(yr + 32 * ks), y_1 = X::row(yr + 16 * LDY + 32 * ks);
            acc[0] = X::mma(y_0, x_0, acc[0]);
            acc[1] = PT::kRev ? X::mma(y_1, x_0, acc[1]) : X::mma(y_0, x_1, acc[1]);
            acc[2] = X::mma(y_1, x_1, acc[2]);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const Frag x_0 = X::row(xr + 32 * ks);
            acc[0] = X::mma(X::row(yr + 32 * ks), x_0, acc[0]);
            acc[1] = X::mma(X::row(yr + 16 * LDY + 32 * ks), x_0, acc[1]);
          }
        }
      };
      if (forms_p) tiles(xrow, yrow, p);
      // p of rows xo + c of x and yo + 4 gq .. of y, decayed; masked: only pairs in order
      const auto decayed = [&](f32x4 v, int xo, int yo, bool masked) {
        const float xh = g_hi[xo + c], xl = g_lo[xo + c];
        const f32x4 yh = lds_f32x4(g_hi + yo + 4 * gq), yl = lds_f32x4(g_lo + yo + 4 * gq);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = PT::kRev ? (yh[j] - xh) + (yl[j] - xl) : (xh - yh[j]) + (xl - yl[j]);
          v[j] = s_p * (v[j] * exp2_fast(e));
          if (masked) v[j] = kept(v[j], PT::kRev ? c - (4 * gq + j) : 4 * gq + j - c);
        }
        return v;
      };
      if (forms_p && diag) {
        p[0] = decayed(p[0], xb, yb, true);
        p[1] = decayed(p[1], PT::kRev ? xb : xb + 16, PT::kRev ? yb + 16 : yb, false);
        p[2] = decayed(p[2], xb + 16, yb + 16, true);
      } else if (forms_p) {
        p[0] = decayed(p[0], xb, yb, false);
        p[1] = decayed(p[1], xb, yb + 16, false);
      }
      if (PASS == kLinDq && forms_p) {  // pairs strictly apart: (q . k) (do . v) decayed, by rows and columns
        f32x4 m[3];
        sched_fence();
        tiles(wrow, zrow, m);
        f32x4 cs[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float m0 = m[0][j] * p[0][j], m1 = m[1][j] * p[1][j];
          if (diag) {
            const int d = 4 * gq + j - c + 1;
            const float a0 = kept(m0, d), a2 = kept(m[2][j] * p[2][j], d);
            r_sum[0] += a0, r_sum[1] += m1 + a2;
            cs[0][j] = a0 + m1, cs[1][j] = a2;
          } else {
            r_sum[0] += m0 + m1;
            cs[0][j] = m0, cs[1][j] = m1;
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) cs[k][j] = row16_sum_dpp(cs[k][j]);
        if (c == 0) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<f32x4 *>(&csum[par][w][16 * k + 4 * gq]) = cs[k];
        }
        const float half = halves_sum(r_sum[0], r_sum[1]), sum = rows_sum(half, half);
        if (gq == 0) rsum[par][w & 1][xb + c] = sum;
        if (gq == 2 && diag) rsum[par][0][xb + 16 + c] = sum;
      }
      const auto store_tile = [&](int xt, int yt, f32x4 v) {
        E *const to = tp + (p_slot<PT::kRev>(xt, yt) * kPTerms * 64 + lane) * 4;
        store4(to, v);
        if (kPTerms == 2) {
          f32x4 unused = zero4();
          X::residual(X::round(v, unused), v, unused);
          store4(to + 256, v);
        }
      };
      const auto store_p = [&]() {
        const int xt = xb / 16, yt = yb / 16;
        store_tile(xt, yt, p[0]);
        if (diag) {
          store_tile(PT::kRev ? xt : xt + 1, PT::kRev ? yt + 1 : yt, p[1]);
          store_tile(xt + 1, yt + 1, p[2]);
          store_tile(PT::kRev ? xt + 1 : xt, PT::kRev ? yt : yt + 1, zero4());
        } else {
          store_tile(xt, yt + 1, p[1]);
        }
      };
      if (!PT::kDots && forms_p) store_p();

      // the state's share: 32 rows of the state at a time, split once for the four row tiles, with
      // the next 32 rows' operands read during the products
#pragma unroll
      for (int xt = 0; xt < 4; ++xt)
#pragma unroll
        for (int t = 0; t < NT; ++t) o[xt][t] = zero4();
      constexpr int XB = PT::kDots ? 1 : 2;  // sets of operands (four tiles leave registers for one)
      Frag xf[XB][4];
      const auto read_x = [&](int ks) {
#pragma unroll
        for (int xt = 0; xt < 4; ++xt) xf[ks % XB][xt] = X::row(tx + (16 * xt + c) * LDX + 32 * ks + 4 * gq);
      };
      sched_fence();
      read_x(0);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if (XB == 2 && ks + 1 < KS) read_x(ks + 1);
        if (XB == 1 && ks > 0) read_x(ks);
        f32x4 s0[NT], s1[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) s0[t] = S[2 * ks][t], s1[t] = S[2 * ks + 1][t];
#pragma unroll
        for (int i = 0; i < kStateTerms; ++i) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const Frag sf = X::round(s0[t], s1[t]);
#pragma unroll
            for (int xt = 0; xt < 4; ++xt) o[xt][t] = X::mma(sf, xf[ks % XB][xt], o[xt][t]);
            if (i + 1 < kStateTerms) X::residual(sf, s0[t], s1[t]);
          }
        }
        sched_fence();
      }
      float d_sum[4];
#pragma unroll
      for (int xt = 0; xt < 4; ++xt) {
        const int xr = 16 * xt + c;
        const float f = f_x[xr];
#pragma unroll
        for (int t = 0; t < NT; ++t) o[xt][t] *= f;
        if (PT::kDots) {  // x's share of dg: w . (the state's share of the output)
          float d = 0.f;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const f32x4 wv = load4(tw + xr * LDX + out_col + 4 * t);
#pragma unroll
            for (int j = 0; j < 4; ++j) d += wv[j] * o[xt][t][j];
          }
          d_sum[xt] = d;
        }
      }
      if (PT::kDots)  // rows of lanes 0 to 3: row tiles 0, 2, 1, 3
        dots[par][w][32 * (gq & 1) + 16 * (gq >> 1) + c] =
            rows_sum(halves_sum(d_sum[0], d_sum[1]), halves_sum(d_sum[2], d_sum[3]));
      read_z();
      lds_barrier();
      if (PT::kDots) {
        if (forms_p) store_p();
        if (it + 1 < nsteps) fetch(in, ch + step);
        lds_barrier();
      }

      // the pairs' share, by 32 rows of y and term; the next operands are read during the products
      Frag pf[XB][4];
      const auto needed = [](int kb, int xt) { return PT::kRev ? 2 * kb + 1 >= xt : 2 * kb <= xt; };
      const auto read_p = [&](int g) {
        const int kb = g / kPTerms, i = g % kPTerms;
#pragma unroll
        for (int xt = 0; xt < 4; ++xt)
          if (needed(kb, xt))
            pf[g % XB][xt] = X::pair(tp + ((p_slot<PT::kRev>(xt, 2 * kb) * kPTerms + i) * 64 + lane) * 4,
                                    kPTerms * 256);
      };
      read_p(0);
#pragma unroll
      for (int g = 0; g < 2 * kPTerms; ++g) {
        if (XB == 2 && g + 1 < 2 * kPTerms) read_p(g + 1);
        if (XB == 1 && g > 0) read_p(g);
#pragma unroll
        for (int xt = 0; xt < 4; ++xt)
          if (needed(g / kPTerms, xt))
#pragma unroll
            for (int t = 0; t < NT; ++t) o[xt][t] = X::mma(zf[g / kPTerms][t], pf[g % XB][xt], o[xt][t]);
        sched_fence();
      }
    }

    // the state after the chunk: by 32 rows of y and z, two 16-row tiles of the state at a time
    const float decay = s_decay[par];
    Frag yf[2][2];
    const auto read_y = [&](int g) {
      const int kb = g / (MT / 2), m = g % (MT / 2) * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        yf[g & 1][i] = X::template column<LDY>(ty + 32 * kb * LDY + 16 * (m + i), y_at);
    };
    read_y(0);

    if constexpr (!PT::kSum) {
      const int n_rows = (int)(t_end - t0 < kChunk ? t_end - t0 : kChunk);
      const auto rsrc = rows_of(out, t0, out_heads, out_head, n_rows, f32_out ? 4 : (int)sizeof(E));
      int c_row = c;
      asm("" : "+v"(c_row));
      const int v_row = c_row * out_heads * D + out_col;
#pragma unroll
      for (int xt = 0; xt < 4; ++xt) {
        const int at = v_row + 16 * xt * out_heads * D;
        if (f32_out || !kB) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o[xt][t]), rsrc, (at + 4 * t) * 4, 0, 0);
        } else if (NT == 2) {
          __builtin_amdgcn_raw_buffer_store_b128(
              __builtin_bit_cast(u32x4, to_bf16x8(o[xt][0], o[xt][NT - 1])), rsrc, at * 2, 0, 0);
        } else {
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, to_bf16x4(o[xt][0])), rsrc, at * 2, 0, 0);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) S[m][t] *= decay;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const f32x4 fa = lds_f32x4(f_y + 32 * kb + 4 * gq), fb = lds_f32x4(f_y + 32 * kb + 16 + 4 * gq);
      if constexpr (PT::kSum && kSets == 1) {  // here: fewer registers through the round
#pragma unroll
        for (int t = 0; t < NT; ++t) zf[kb][t] = X::template column<LDY>(tz + 32 * kb * LDY + 4 * t, z_at);
      }
      Frag b1[NT], b2[NT], b3[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4 u = fa * X::lo_part(zf[kb][t]), v = fb * X::hi_part(zf[kb][t]);
        b1[t] = X::round(u, v);
        if constexpr (kB) {
          X::residual(b1[t], u, v);
          b2[t] = X::round(u, v);
          if (precise) {
            X::residual(b2[t], u, v);
            b3[t] = X::round(u, v);
          }
        }
      }
#pragma unroll
      for (int mm = 0; mm < MT / 2; ++mm) {
        const int g = kb * (MT / 2) + mm, m = 2 * mm;
        if (g + 1 < MT) read_y(g + 1);
        const auto add = [&](const Frag(&b)[NT]) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) S[m + i][t] = X::mma(yf[g & 1][i], b[t], S[m + i][t]);
        };
        add(b1);
        if constexpr (kB) {
          add(b2);
          if (precise) add(b3);
        }
        sched_fence();
      }
    }
    if (w == kDecayWave && it + 1 < nsteps) make_decays(next.g, par ^ 1);
  };
  for (int it = 0; it < nsteps; it += kSets, ch += step) {
    round(it, set[0], set[kSets - 1]);
    if (kSets > 1 && it + 1 < nsteps) {
      ch += step;
      round(it + 1, set[kSets - 1], set[0]);
    }
  }
  if (PT::kDots && nsteps > 0) {
    __syncthreads();
    flush_dots(ch - step, (nsteps - 1) & 1);
  }

  // the same column, made anew: not a register through all rounds
  int c_end = lane & 15;
  asm("" : "+v"(c_end));
  const int col_end = NT == 2 ? 32 * w + 8 * (c_end >> 2) + (c_end & 3) : 16 * w + c_end;
  const auto store_state = [&](float *to) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) to[(16 * m + 4 * gq + j) * D + col_end + 4 * t] = S[m][t][j];
  };
  if (PT::kSum) {
    store_state((PT::kRev ? a.unit_r : a.unit_s) + uh * D * D);
    if (w == kDecayWave && lane == 0)
      a.unit_decay[(PT::kRev ? a.units * a.H : 0) + uh] = exp2_fast(total.hi + total.lo);
  }
  if ((PASS == kLinFwd || PASS == kLinDv) && edge_out && final_state)
    store_state(final_state + ((int64_t)seq * a.H + h) * D * D);
  if (PASS == kLinDq) {  // <state, its gradient> at the unit's end
    const float *ds = last ? (a.dht ? a.dht + ((int64_t)seq * a.H + h) * D * D : nullptr)
                           : a.unit_r + uh * D * D;
    double d = 0.0;
    if (ds) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const f32x4 x = *reinterpret_cast<const f32x4 *>(ds + (col_end + 4 * t) * D + 16 * m + 4 * gq);
          float s = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) s += x[j] * S[m][t][j];
          d += s;
        }
    }
    d = wave_sum_f64(d);
    __syncthreads();  // the last chunk's parts have been read
    if (lane == 0) dots[0][w][0] = (float)d;
    __syncthreads();
    if (tid == 0) {
      float sum = dots[0][0][0];
#pragma unroll
      for (int i = 1; i < WAVES; ++i) sum += dots[0][i][0];
      a.unit_dot[uh] = sum;
    }
  }
}

// One pass, or (GROUP) the passes of one stage of the backward side by side: grid z picks it.
// kGroupSums: the units' sums in both directions; kGroupGrads: dq, dk, dv.
enum { kGroupSums = 16, kGroupGrads };

template <class E, int D, int WHAT>
constexpr size_t stage_lds_bytes() {
  if constexpr (WHAT == kGroupSums) {
    return pass_lds_bytes<E, D, kLinSumFwd>();
  } else if constexpr (WHAT == kGroupGrads) {
    return std::max(pass_lds_bytes<E, D, kLinDq>(), pass_lds_bytes<E, D, kLinDv>());
  } else {
    return pass_lds_bytes<E, D, WHAT>();
  }
}

// Three workgroups per CU: the forward's sums of d = 128, with one chunk's rows on their way (32K
// tokens x 8 heads, whole forward: 142 to 137 us).  Those of the backward, twice as many units at
// once, are faster two by two with two chunks' rows each (65K tokens: 660 against 674 us).
template <class E, int D, int WHAT, int WAVES>
constexpr bool kThree = sizeof(E) == 2 && D == 128 && WHAT == kLinSumFwd && WAVES == 4;

template <class E, int D, int WHAT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, (kThree<E, D, WHAT, WAVES> ? 3 : sizeof(E) == 2 || WAVES == 8 ? 2 : 1)) void lin_stage_kernel(LinArgs a) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ PassShared<WAVES> sh;
  if constexpr (WHAT == kGroupSums) {
    if (blockIdx.z == 0) lin_pass<E, D, kLinSumFwd, WAVES, 2>(a, smem, sh);
    else lin_pass<E, D, kLinSumRev, WAVES, 2>(a, smem, sh);
  } else if constexpr (WHAT == kGroupGrads) {
    if (blockIdx.z == 0) lin_pass<E, D, kLinDq, WAVES, 1>(a, smem, sh);
    else if (blockIdx.z == 1) lin_pass<E, D, kLinDk, WAVES, 1>(a, smem, sh);
    else lin_pass<E, D, kLinDv, WAVES, 1>(a, smem, sh);
  } else {
    lin_pass<E, D, WHAT, WAVES, (kThree<E, D, WHAT, WAVES> || WHAT != kLinSumFwd ? 1 : 2)>(a, smem, sh);
  }
}

namespace {

// The states at the units' starts from the units' own sums, in place: along each sequence of more
// than one unit, S <- decay_u S + sum_u, written where unit u + 1's sum was.  rev: the gradients at
// the units' ends, from the last unit to the first.  One thread per four elements of a state, its
// loads kAhead units ahead of the chain: a chain's step is a few instructions, so the time is that
// of the bytes in flight (65K tokens x 8 heads, both directions, 124 MB: 21 us, 5.8 TB/s; one chain
// of 57 units x 8 heads, 59 MB: 21 us, 2.8 TB/s; 32 units ahead change neither).
constexpr int kAhead = 16, kScanThreads = 128;

template <bool REV>
__device__ __forceinline__ void lin_scan(const LinArgs &a, int D, int64_t e) {
  const int seq = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 63;
  const int64_t DD = (int64_t)D * D;
  const int32_t b0 = __builtin_amdgcn_readfirstlane(a.cu[seq]), b1 = __builtin_amdgcn_readfirstlane(a.cu[seq + 1]);
  if (b0 < 0 || b1 < b0 || b1 > a.T) return;
  const int nch = (b1 - b0 + kChunk - 1) / kChunk, nu = (nch + a.L - 1) / a.L;
  if (nu < 2) return;
  const int64_t u0 = __builtin_amdgcn_readfirstlane(a.seq_unit[seq]);
  if (u0 < 0 || u0 + nu > a.units) return;  // a malformed table gave this sequence no units
  const int64_t row = (int64_t)a.H * DD;
  float *const st = (REV ? a.unit_r : a.unit_s) + u0 * row + h * DD + e;
  const float *const dec = a.unit_decay + (REV ? a.units * a.H : 0) + u0 * a.H + h;
  f32x4 S = zero4();
  const float *init = REV ? (a.dht ? a.dht + ((int64_t)seq * a.H + h) * DD + e : nullptr)
                          : (a.h0 ? a.h0 + seq * a.h0_stride + h * DD + e : nullptr);
  if (init) S = *reinterpret_cast<const f32x4 *>(init);
  // step s passes unit us(s) and writes the state to unit us(s + 1), whose sum was read kAhead
  // steps before its own step, so always before that write
  const int steps = nu - 1;
  const auto us = [&](int s) { return REV ? nu - 1 - s : s; };
  f32x4 b[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (j < steps) b[j] = *reinterpret_cast<const f32x4 *>(st + us(j) * row);
  for (int s64 = 0; s64 < steps; s64 += 64) {  // 64 units' decays, one in each lane
    const float dl = s64 + lane < steps ? dec[(int64_t)us(s64 + lane) * a.H] : 0.f;
    const int end = min(steps, s64 + 64);
    for (int s0 = s64; s0 < end; s0 += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int s = s0 + j;
        if (s < end) {
          const float d = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(dl), s & 63));
          S = d * S + b[j];
          if (s + kAhead < steps) b[j] = *reinterpret_cast<const f32x4 *>(st + us(s + kAhead) * row);
          *reinterpret_cast<f32x4 *>(st + us(s + 1) * row) = S;
        }
      }
    }
  }
}

// grid z: D^2 / 512 pieces of the states, then (both directions) as many of the state gradients
__global__ __launch_bounds__(kScanThreads) void lin_scan_kernel(LinArgs a, int D) {
  const int pieces = D * D / (4 * kScanThreads), z = blockIdx.z;
  const int64_t e = ((int64_t)(z < pieces ? z : z - pieces) * kScanThreads + threadIdx.x) * 4;
  if (z < pieces) lin_scan<false>(a, D, e);
  else lin_scan<true>(a, D, e);
}

// dg_t = <dS_t, e^{g_t} S_{t-1}> from its parts: the pairs within the chunk on both sides of t,
// and the scan of q . dq and k . dk (the states' shares) from the unit's end, where
// <S, dS> is known: sum_{s >= t} (q_s . dq_s - k_s . dk_s) + <S, dS>_end.  Both parts are
// differences (the pairs' of row and column sums), so dg's error is absolute: fp32's rounding of the
// |q_s . dq_s| and |k_s . dk_s| of the unit, from whose end the scan starts anew.  The sums themselves
// are pairs of floats and add nothing to it.  One workgroup per (unit, head), from the unit's end by blocks of 64 chunks: the waves
// sum their chunks side by side, then finish them with the sums of the later ones.  A token whose
// decay is zero in fp32 has no gradient.  (65K tokens x 8 heads: 17 us.)
__device__ __forceinline__ F2 lane_of(F2 x, int l) {
  return F2{__shfl(x.hi, l, 64), __shfl(x.lo, l, 64)};
}
// ... of a lane that is the same for the whole wave (and may be inactive)
__device__ __forceinline__ F2 lane_of_uniform(F2 x, int l) {
  return F2{__int_as_float(__builtin_amdgcn_readlane(__float_as_int(x.hi), l)),
            __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x.lo), l))};
}

__global__ __launch_bounds__(256) void lin_dg_kernel(LinArgs a) {
  __shared__ F2 sums[64];
  __shared__ double part[4];
  __shared__ int sh_unit[3];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, h = blockIdx.y;
  const int64_t uh = (int64_t)blockIdx.x * a.H + h;
  if (w == 0) {
    Unit un{};
    const bool ok = find_unit(a.cu, a.N, a.T, a.L, blockIdx.x, false, lane, un);
    if (lane == 0) {
      sh_unit[0] = ok ? un.seq : -1;
      sh_unit[1] = un.c0;
      sh_unit[2] = un.c1;
    }
  }
  __syncthreads();
  const int seq = sh_unit[0], c0 = sh_unit[1], c1 = sh_unit[2];
  const int64_t t_beg = seq < 0 ? 0 : a.cu[seq], t_end = seq < 0 ? 0 : a.cu[seq + 1];
  const bool ok = seq >= 0 && t_beg >= 0 && t_end >= t_beg && t_end <= a.T && c1 > c0;
  double total = 0.0;
  if (ok) {
    const float *const dq = a.dg_q + (int64_t)h * a.T, *const dk = a.dg_k + (int64_t)h * a.T;
    const float *const pairs = a.dg_pairs + (int64_t)h * a.T;
    F2 b = F2{a.unit_dot[uh], 0.f};  // <S, dS> at the end of the block
    const float gh = a.g_head ? a.g[h] : 0.f;
    // x and the later lanes' x: the wave's sum less the sum before
    const auto from_here = [&](F2 x, F2 &all) {
      const F2 up = wave_scan2(x);
      all = lane_of(up, 63);
      return add2(add2(all, F2{-up.hi, -up.lo}), x);
    };
    for (int hi = c1; hi > c0; hi -= 64) {  // chunks [lo, hi)
      const int lo = max(c0, hi - 64), n = hi - lo;
      for (int j = w; j < n; j += 4) {
        const int64_t t = t_beg + (int64_t)(lo + j) * kChunk + lane;
        F2 all;
        from_here(t < t_end ? add2(F2{dq[t], 0.f}, F2{-dk[t], 0.f}) : F2{0.f, 0.f}, all);
        if (lane == 0) sums[j] = all;
      }
      __syncthreads();
      // lane j: the sum of the block's chunks after chunk j
      const F2 x = lane < n ? sums[lane] : F2{0.f, 0.f};
      F2 whole;
      const F2 after = add2(from_here(x, whole), F2{-x.hi, -x.lo});
      for (int j = w; j < n; j += 4) {
        const int64_t t = t_beg + (int64_t)(lo + j) * kChunk + lane;
        const bool in = t < t_end;
        F2 all;
        const F2 s = from_here(in ? add2(F2{dq[t], 0.f}, F2{-dk[t], 0.f}) : F2{0.f, 0.f}, all);
        if (in) {
          const F2 lg = log2_decay(a.g_head ? gh : a.g[t * a.H + h]);
          F2 dg = add2(add2(add2(b, lane_of_uniform(after, j)), s), F2{pairs[t], 0.f});
          if (lg.hi <= kNoDecay) dg = F2{0.f, 0.f};
          if (!a.g_head) a.dg[t * a.H + h] = dg.hi + dg.lo;
          total += (double)dg.hi + (double)dg.lo;
        }
      }
      b = add2(b, whole);
      __syncthreads();
    }
  }
  if (a.g_head) {
    total = wave_sum_f64(total);
    if (lane == 0) part[w] = total;
    __syncthreads();
    if (threadIdx.x == 0) a.dg_unit[uh] = part[0] + part[1] + part[2] + part[3];
  }
}

// dg of each head's constant decay: the units' sums, in a fixed order.
__global__ __launch_bounds__(256) void lin_dg_head_kernel(LinArgs a) {
  __shared__ double part[4];
  const int h = blockIdx.x;
  double s = 0.0;
  for (int64_t u = threadIdx.x; u < a.units; u += 256) s += a.dg_unit[u * a.H + h];
  s = wave_sum_f64(s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) a.dg[h] = (float)(part[0] + part[1] + part[2] + part[3]);
}

// dq (grid y = 0) and dk of key heads from their value heads' shares.
template <class E>
__global__ __launch_bounds__(256) void lin_group_sum_kernel(LinArgs a, int D4, E *dq, E *dk) {
  const float *const part = static_cast<const float *>(blockIdx.y == 0 ? a.dq : a.dk);
  E *const out = blockIdx.y == 0 ? dq : dk;
  const int G = a.H / a.HK;
  // rows of no sequence have no parts and stay as they are
  const int64_t row = (int64_t)a.HK * D4, i1 = min((int64_t)a.cu[a.N], a.T) * row;
  for (int64_t i = max(a.cu[0], 0) * row + (int64_t)blockIdx.x * 256 + threadIdx.x; i < i1;
       i += (int64_t)gridDim.x * 256) {
    const f32x4 *p = reinterpret_cast<const f32x4 *>(part) + i / D4 * G * D4 + i % D4;
    f32x4 s = p[0];
    for (int j = 1; j < G; ++j) s += p[(int64_t)j * D4];
    store4(out + 4 * i, s);
  }
}

__global__ __launch_bounds__(256) void lin_zero_kernel(float *x, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    x[i] = 0.f;
}

template <class E, int D, int WHAT, int WAVES>
hipError_t launch_stage(const LinArgs &a, int kinds, hipStream_t stream) {
  constexpr size_t lds = stage_lds_bytes<E, D, WHAT>();
  if (lds > 65536) {  // above the default limit of dynamic LDS, which is raised once per device
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = (uint64_t)1 << (dev & 63);
    if (dev > 63 || !(raised.load(std::memory_order_relaxed) & bit)) {
      e = hipFuncSetAttribute(reinterpret_cast<const void *>(&lin_stage_kernel<E, D, WHAT, WAVES>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
      if (e != hipSuccess) return e;
      if (dev <= 63) raised.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  const unsigned u = (unsigned)a.units, h = (unsigned)a.H;
  hipLaunchKernelGGL((lin_stage_kernel<E, D, WHAT, WAVES>),
                     a.longest_first ? dim3(h, u, kinds) : dim3(u, h, kinds), dim3(64 * WAVES), lds,
                     stream, a);
  return hipGetLastError();
}

// Waves per workgroup, d = 128: a workgroup that has a CU to itself takes eight, with 16 columns of
// the state each (8K packed tokens x 8 heads, 237 workgroups: 71 to 60 us; fp32, 2K tokens, backward:
// 79 to 72 us, always alone on its CU); where two of four waves share a CU eight are slower (65K
// tokens, backward: 663 against 753 us), since P is still formed by four.
template <class E, int D, int WHAT>
hipError_t launch_stage(const LinArgs &a, hipStream_t stream) {
  constexpr int kinds = WHAT == kGroupSums ? 2 : WHAT == kGroupGrads ? 3 : 1;
  if constexpr (D == 64) {
    return launch_stage<E, D, WHAT, 4>(a, kinds, stream);
  } else if constexpr (sizeof(E) == 4) {
    return launch_stage<E, D, WHAT, 8>(a, kinds, stream);
  } else {
    // about that many: the last unit of a sequence is on average half a unit
    const int64_t units = a.L > 0 ? (a.T / kChunk) / a.L + (a.N + 1) / 2 : a.N;
    return units * a.H * kinds <= a.cus ? launch_stage<E, D, WHAT, 8>(a, kinds, stream)
                                        : launch_stage<E, D, WHAT, 4>(a, kinds, stream);
  }
}

template <int WHAT>
hipError_t launch_stage_of(const LinArgs &a, int D, bool is_bf16, hipStream_t stream) {
  if (D == 128)
    return is_bf16 ? launch_stage<bf16, 128, WHAT>(a, stream) : launch_stage<float, 128, WHAT>(a, stream);
  return is_bf16 ? launch_stage<bf16, 64, WHAT>(a, stream) : launch_stage<float, 64, WHAT>(a, stream);
}

hipError_t launch_scan(const LinArgs &a, int D, int directions, hipStream_t stream) {
  hipLaunchKernelGGL(lin_scan_kernel, dim3((unsigned)a.N, a.H, directions * (D * D / (4 * kScanThreads))),
                     dim3(kScanThreads), 0,
                     stream, a, D);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linattn_fwd(const LinArgs &a, int D, bool is_bf16, hipStream_t stream) {
  if (a.L > 0) {
    hipError_t e = launch_stage_of<kLinSumFwd>(a, D, is_bf16, stream);
    if (e == hipSuccess) e = launch_scan(a, D, 1, stream);
    if (e != hipSuccess) return e;
  }
  return launch_stage_of<kLinFwd>(a, D, is_bf16, stream);
}

hipError_t launch_linattn_bwd(const LinArgs &a, int D, bool is_bf16, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.L > 0) {
    e = launch_stage_of<kGroupSums>(a, D, is_bf16, stream);
    if (e == hipSuccess) e = launch_scan(a, D, 2, stream);
    if (e != hipSuccess) return e;
  }
  e = launch_stage_of<kGroupGrads>(a, D, is_bf16, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(lin_dg_kernel, dim3((unsigned)a.units, a.H), dim3(256), 0, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess || !a.g_head) return e;
  hipLaunchKernelGGL(lin_dg_head_kernel, dim3(a.H), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_linattn_group_sum(const LinArgs &a, int D, bool is_bf16, void *dq, void *dk,
                                    hipStream_t stream) {
  const int64_t n4 = a.T * a.HK * D / 4;
  if (n4 <= 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>((n4 + 255) / 256, 16384), 2);
  if (is_bf16)
    hipLaunchKernelGGL(lin_group_sum_kernel<bf16>, grid, dim3(256), 0, stream, a, D / 4,
                       static_cast<bf16 *>(dq), static_cast<bf16 *>(dk));
  else
    hipLaunchKernelGGL(lin_group_sum_kernel<float>, grid, dim3(256), 0, stream, a, D / 4,
                       static_cast<float *>(dq), static_cast<float *>(dk));
  return hipGetLastError();
}

hipError_t launch_linattn_zero(float *x, int64_t n, hipStream_t stream) {
  hipLaunchKernelGGL(lin_zero_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 1024)),
                     dim3(256), 0, stream, x, n);
  return hipGetLastError();
}

}  // namespace gdn
