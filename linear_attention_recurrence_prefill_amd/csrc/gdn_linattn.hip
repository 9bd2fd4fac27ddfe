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
// (lin_scan_kernel), the unit run from its true start.
//
// Work of one workgroup (256 threads, 4 waves): one (unit, head).  Wave w owns D / 4 columns of the
// state, all D rows of them, in MFMA accumulators: in that layout (lane n + 16 (m / 4), item m % 4)
// two stacked 16-row tiles are, as they stand, the operand of a 16x16x32 product over the rows, in
// the row order {4 gq + j, 16 + 4 gq + j}.  All row operands are read in that order, so neither
// the state nor the 64 x 64 products P ever pass through LDS, and waves meet only at the tile
// buffers.  P is formed by every wave (40 of its some 200 MFMAs per chunk).  Output tiles are
// formed transposed (columns by items), so a lane stores 16 consecutive bytes of a row.
//
// Rounding: inputs are bf16, sums and states fp32.  Products take bf16 operands; what is not an
// input is split into a sum of bf16 terms: two terms (2^-17) where the result is rounded to bf16
// in the end, three (2^-25) where it is kept in fp32 (final states, state gradients, dg's parts).
// fp32 inputs use the fp32 MFMA throughout.
//
// Decays: G in units of log2, accumulated as a pair of floats (hi + lo), and only differences of G
// are exponentiated, so no factor overflows and far tokens keep their precision.  Log decays below
// kMinLog2 have no fp32 value above zero and are taken as kMinLog2: -inf empties the state.
#include <algorithm>

#include "gdn_device.h"
#include "gdn_internal.h"
#include "gdn_linattn.h"
#include "gdn_unit.h"

namespace gdn {
namespace {

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
// bf16 tiles: rows of D + 16 elements (8 (mod 64) banks apart), and in every other group of eight
// rows the 16-byte units are exchanged in pairs.  The eight rows that a half wave's transposing
// read takes then lie on different banks, and so do the sixteen rows of a row read.
template <>
struct Op<bf16> {
  typedef bf16x8 Frag;
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  static constexpr int kPad = 16;
  // where column `col` of row `row` is within the row (col in units that stay whole: 4 elements)
  static __device__ __forceinline__ int place(int row, int col) { return col ^ (row & 8); }
  static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) { return mma_bf16(a, b, c); }
  // a row, from its element at index 4 gq on (a multiple of 32 further: the next products')
  static __device__ __forceinline__ Frag row(const bf16 *p) {
    return cat8(lds_bf16x4(p), lds_bf16x4(p + 16));
  }
  // a column: rows row0 + (order) of column `col`; `colq` is the column this lane addresses
  template <int LD>
  static __device__ __forceinline__ Frag column(const bf16 *tile, int row0, int colq, int, int c,
                                                int gq) {
    const int r = 4 * gq + (c >> 2);
    const bf16 *p = tile + (row0 + r) * LD + place(r, colq);
    return cat8(lds_tr16(p), lds_tr16(p + 16 * LD));
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
  static constexpr int kPad = 4;
  static __device__ __forceinline__ int place(int, int col) { return col; }
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
  template <int LD>
  static __device__ __forceinline__ Frag column(const float *tile, int row0, int, int col, int,
                                                int gq) {
    const float *p = tile + (row0 + 4 * gq) * LD + col;
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
__device__ __forceinline__ void store8(float *p, f32x4 x, f32x4 y) {
  store4(p, x);
  store4(p + 4, y);
}
__device__ __forceinline__ void store8(bf16 *p, f32x4 x, f32x4 y) {
  *reinterpret_cast<bf16x8 *>(p) = to_bf16x8(x, y);
}

__device__ __forceinline__ f32x4 load4(const bf16 *p) {
  const bf16x4 x = lds_bf16x4(p);
  return f32x4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
}
__device__ __forceinline__ f32x4 load4(const float *p) { return lds_f32x4(p); }

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
  const size_t tile = (size_t)64 * (D + Op<E>::kPad) * sizeof(E);
  return PT::kTiles * tile + (PT::kSum || PT::kDots ? 0 : p_bytes<E>());
}

}  // namespace

template <class E, int D, int PASS>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 2 : 1) void lin_pass_kernel(LinArgs a) {
  typedef Op<E> X;
  typedef typename X::Frag Frag;
  typedef PassTraits<PASS> PT;
  constexpr int LD = D + X::kPad;
  constexpr int NT = D / 64;      // 16-column tiles of the state per wave
  constexpr int MT = D / 16;      // 16-row tiles of the state
  constexpr int KS = D / 32;      // products over a row
  constexpr int EPU = 16 / (int)sizeof(E);
  constexpr int UPR = D / EPU;            // 16-byte units per row
  constexpr int UPT = 64 * UPR / 256;     // ... per thread and tile
  // terms of the split operands (see the file's head)
  constexpr bool kB = sizeof(E) == 2;
  constexpr int kStateTerms = !kB ? 1 : (PT::kDots ? 3 : 2);
  constexpr int kPTerms = p_terms<E>();
  constexpr int kDecayWave = PT::kRev ? 3 : 0;  // the wave with the fewest tiles of P

  extern __shared__ __attribute__((aligned(16))) char smem[];
  E *const ty = reinterpret_cast<E *>(smem);   // tiles [64][LD]: y, z, x, w
  E *const tz = ty + 64 * LD;
  E *const tx = tz + 64 * LD;
  E *const tw = tx + 64 * LD;
  // P: behind the tiles, or (four tiles) over x, which is dead by then
  E *const tp = PT::kDots ? tx : tx + 64 * LD;
  __shared__ __attribute__((aligned(16))) float g_hi[64], g_lo[64], f_x[64], f_y[64], f_a[64], f_b[64];
  __shared__ float sh_decay;
  __shared__ float dots[2][4][64], rsum[2][64], csum[2][4][64];  // by the chunk's parity
  __shared__ int sh_unit[4];

  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, gq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.y, hk = h / (a.H / a.HK);

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
  const int seq = __builtin_amdgcn_readfirstlane(sh_unit[0]);
  const int c0 = __builtin_amdgcn_readfirstlane(sh_unit[1]);
  const int c1 = __builtin_amdgcn_readfirstlane(sh_unit[2]);
  if (seq < 0) return;
  const int64_t t_beg = a.cu[seq], t_end = a.cu[seq + 1];
  if (t_beg < 0 || t_end < t_beg || t_end > a.T) return;
  const int nch = (int)((t_end - t_beg + kChunk - 1) / kChunk);
  const bool first = c0 == 0, last = c1 >= nch;
  const bool edge_in = PT::kRev ? last : first;    // the pass starts at the sequence's edge
  const bool edge_out = PT::kRev ? first : last;   // ... ends there
  const int64_t uh = (int64_t)blockIdx.x * a.H + h;
  if (PT::kSum) {
    if (PASS == kLinSumFwd && first && h == 0 && tid == 0) a.seq_unit[seq] = blockIdx.x;
    if (edge_out) return;  // no unit follows
  }

  // the rows of this pass
  const void *px = nullptr, *py, *pz, *pw = nullptr;
  int hx = h, hy = h, hz = h, nx = a.H, ny = a.H, nz = a.H;
  if (PASS == kLinFwd) {
    px = a.q, py = a.k, pz = a.v, hx = hy = hk, nx = ny = a.HK;
  } else if (PASS == kLinDq) {
    px = a.dout, py = a.v, pz = a.k, pw = a.q, hz = hk, nz = a.HK;
  } else if (PASS == kLinDv) {
    px = a.k, py = a.q, pz = a.dout, hx = hy = hk, nx = ny = a.HK;
  } else if (PASS == kLinDk) {
    px = a.v, py = a.dout, pz = a.q, pw = a.k, hz = hk, nz = a.HK;
  } else if (PASS == kLinSumFwd) {
    py = a.k, pz = a.v, hy = hk, ny = a.HK;
  } else {
    py = a.q, pz = a.dout, hy = hk, ny = a.HK;
  }
  const float s_out = PASS == kLinFwd || PASS == kLinDq ? a.scale : 1.f;
  const float s_in = PT::kRev ? a.scale : 1.f;

  // this wave's columns of the state: tile t's column of lane c, and the column that lane c
  // addresses in a transposing read
  int col[NT], colq[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    col[t] = NT == 2 ? 32 * w + 8 * (c >> 2) + 4 * t + (c & 3) : 16 * w + c;
    colq[t] = NT == 2 ? 32 * w + 8 * (c & 3) + 4 * t : 16 * w + 4 * (c & 3);
  }
  const int rowq = X::place(c, 4 * gq);  // a row operand's first element (rows 16 i + c)
  const int out_col = NT == 2 ? 32 * w + 8 * gq : 16 * w + 4 * gq;  // first column it stores

  const bool per_k = PT::kDots && !a.out_f32;  // dq, dk of ungrouped heads
  const int out_heads = per_k ? a.HK : a.H, out_head = per_k ? hk : h;
  const int64_t out_size = PT::kDots && a.out_f32 ? 4 : (int64_t)sizeof(E);
  const unsigned v_out = (unsigned)((c * out_heads * D + out_col) * out_size);

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
          S[m][t] = *reinterpret_cast<const f32x4 *>(src + col[t] * D + r);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) S[m][t][j] = src[(r + j) * D + col[t]];
        }
      }
    }

  uint4 sy[UPT], sz[UPT], sx[UPT], sw[UPT];  // the next chunk's rows
  float sg = 0.f;                            // ... log decays (wave 0)
  // addresses: a uniform base per 256 units and one 32-bit offset per lane and row stride
  const int r0 = tid / UPR, o0 = tid % UPR * EPU;
  constexpr int kRows = 256 / UPR;  // rows per 256 units
  const unsigned vx = (unsigned)((r0 * nx * D + o0) * sizeof(E)), vy = (unsigned)((r0 * ny * D + o0) * sizeof(E));
  const unsigned vz = (unsigned)((r0 * nz * D + o0) * sizeof(E)), vw = (unsigned)((r0 * a.HK * D + o0) * sizeof(E));
  const auto load16 = [](const void *base, int64_t elems, unsigned v) {
    return *reinterpret_cast<const uint4 *>(static_cast<const char *>(base) + elems * (int64_t)sizeof(E) + v);
  };
  const auto fetch = [&](int ch) {
    const int64_t t0 = t_beg + (int64_t)ch * kChunk;
    const int n = (int)(t_end - t0 < kChunk ? t_end - t0 : kChunk);
    const auto rows = [&](int u) {
      const int64_t t = t0 + kRows * u;
      sy[u] = load16(py, (t * ny + hy) * D, vy);
      sz[u] = load16(pz, (t * nz + hz) * D, vz);
      if (!PT::kSum) sx[u] = load16(px, (t * nx + hx) * D, vx);
      if (PT::kDots) sw[u] = load16(pw, (t * a.HK + hk) * D, vw);
    };
    if (n == kChunk) {
#pragma unroll
      for (int u = 0; u < UPT; ++u) rows(u);
    } else {
#pragma unroll
      for (int u = 0; u < UPT; ++u) {
        sy[u] = sz[u] = sx[u] = sw[u] = uint4{0u, 0u, 0u, 0u};
        if (r0 + kRows * u < n) rows(u);
      }
    }
    if (w == kDecayWave) sg = lane < n ? a.g[a.g_head ? h : (t0 + lane) * a.H + h] : 0.f;
  };
  // the decays of the chunk that was fetched (one wave), kept in registers until its tiles are up
  F2 G{}, GC{}, total{0.f, 0.f};  // total: the unit's whole log decay
  float from_start = 0.f, to_end = 0.f, near_a = 0.f, near_b = 0.f;
  const auto make_decays = [&]() {
    G = wave_scan2(log2_decay(sg));
    GC = F2{__shfl(G.hi, 63, 64), __shfl(G.lo, 63, 64)};
    from_start = exp2_fast(G.hi + G.lo);
    to_end = exp2_fast((GC.hi - G.hi) + (GC.lo - G.lo));
    if (!PT::kSum) {
      // decay from the end of the 16-token tile before, and to the end of its own
      const int e = lane | 15, b = e < 16 ? 0 : e - 16;
      const F2 E1 = F2{__shfl(G.hi, e, 64), __shfl(G.lo, e, 64)};
      const F2 B1 = F2{__shfl(G.hi, b, 64), __shfl(G.lo, b, 64)};
      near_a = exp2_fast((G.hi - B1.hi) + (G.lo - B1.lo));
      near_b = exp2_fast((E1.hi - G.hi) + (E1.lo - G.lo));
    } else {
      total = add2(total, GC);
    }
  };
  // dg's parts of the chunk before (every wave's share is in LDS)
  const auto flush_dots = [&](int ch, int par) {
    if (!PT::kDots || w != 1) return;
    const int64_t t = t_beg + (int64_t)ch * kChunk + lane;
    float *const to = PASS == kLinDq ? a.dg_q : a.dg_k;
    const float d = dots[par][0][lane] + dots[par][1][lane] + dots[par][2][lane] + dots[par][3][lane];
    if (t < t_end) to[t * a.H + h] = d;
    if (PASS == kLinDq) {
      // sum over the pairs s >= t > i = sum_{s >= t} (row sum - column sum); rows from the end
      F2 x = F2{rsum[par][lane], 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j) x = add2(x, F2{-csum[par][j][lane], 0.f});
      const F2 up = wave_scan2(x);
      const float th = __shfl(up.hi, 63, 64), tl = __shfl(up.lo, 63, 64);
      const F2 rest = add2(add2(F2{th, tl}, F2{-up.hi, -up.lo}), x);
      if (t < t_end) a.dg_pairs[t * a.H + h] = rest.hi + rest.lo;
    }
  };

  const int step = PT::kRev ? -1 : 1;
  int ch = PT::kRev ? c1 - 1 : c0;
  const int nsteps = c1 - c0;
  // terms of the state update: three where the state is written out or feeds dg
  const bool precise = kB && (PT::kSum || PT::kDots || (edge_out && a.final_state != nullptr));
  if (nsteps > 0) {
    fetch(ch);
    if (w == kDecayWave) make_decays();
  }
  for (int it = 0; it < nsteps; ++it, ch += step) {
    const int64_t t0 = t_beg + (int64_t)ch * kChunk;
    __syncthreads();
    const int par = it & 1;
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      const int o = (r0 + kRows * u) * LD + X::place(r0 + kRows * u, o0);
      *reinterpret_cast<uint4 *>(ty + o) = sy[u];
      *reinterpret_cast<uint4 *>(tz + o) = sz[u];
      if (!PT::kSum) *reinterpret_cast<uint4 *>(tx + o) = sx[u];
      if (PT::kDots) *reinterpret_cast<uint4 *>(tw + o) = sw[u];
    }
    if (w == kDecayWave) {
      f_x[lane] = PT::kRev ? to_end : from_start;
      f_y[lane] = PT::kRev ? s_in * from_start : to_end;
      if (!PT::kSum) {
        g_hi[lane] = G.hi;
        g_lo[lane] = G.lo;
        f_a[lane] = near_a;
        f_b[lane] = near_b;
      }
      if (lane == 0) sh_decay = exp2_fast(GC.hi + GC.lo);
    }
    __syncthreads();
    if (it > 0) flush_dots(ch - step, par ^ 1);
    // the next chunk's loads: at once, or (four tiles) once the output's registers are free
    if (!PT::kDots && it + 1 < nsteps) fetch(ch + step);

    f32x4 o[4][NT];  // the output by 16-row tiles
    if constexpr (!PT::kSum) {
      // the pairs within the chunk: wave w forms P's tiles of its 16 rows of x
      f32x4 p[4];
      {
        const int xr = 16 * w + c;
        Frag xf[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) xf[ks] = X::row(tx + xr * LD + rowq + 32 * ks);
        const float xh = g_hi[xr], xl = g_lo[xr], x_near = PT::kRev ? f_b[xr] : f_a[xr];
        // all four tiles of the row, so that every wave runs the same straight line of independent
        // products; the tiles it does not need are dropped
#pragma unroll
        for (int yt = 0; yt < 4; ++yt) p[yt] = zero4();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int yt = 0; yt < 4; ++yt)
            p[yt] = X::mma(X::row(ty + (16 * yt + c) * LD + rowq + 32 * ks), xf[ks], p[yt]);
#pragma unroll
        for (int yt = 0; yt < 4; ++yt) {
          if (PT::kRev ? yt < w : yt > w) {
            p[yt] = zero4();
          } else if (yt != w) {
            // e^{G_late - G_early} = to the end of the earlier tile, the tiles between, and from
            // there: each factor at most one, no exponential per pair
            const int e0 = 16 * (PT::kRev ? w : yt) + 15, e1 = 16 * (PT::kRev ? yt : w) - 1;
            const float mid = exp2_fast((g_hi[e1] - g_hi[e0]) + (g_lo[e1] - g_lo[e0]));
            const float fx = s_in * (x_near * mid);
            const f32x4 fy = lds_f32x4((PT::kRev ? f_a : f_b) + 16 * yt + 4 * gq);
#pragma unroll
            for (int j = 0; j < 4; ++j) p[yt][j] *= fx * fy[j];
          } else {
            const f32x4 yh = lds_f32x4(g_hi + 16 * yt + 4 * gq);
            const f32x4 yl = lds_f32x4(g_lo + 16 * yt + 4 * gq);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int d = 4 * gq + j - c;
              const float e = PT::kRev ? (yh[j] - xh) + (yl[j] - xl) : (xh - yh[j]) + (xl - yl[j]);
              const bool in = PT::kRev ? d >= 0 : d <= 0;
              p[yt][j] = in ? s_in * (p[yt][j] * exp2_fast(e)) : 0.f;
            }
          }
        }
        if (PASS == kLinDq) {  // pairs strictly apart: (q . k) (do . v) decayed
          float r = 0.f;
          Frag qf[KS];
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) qf[ks] = X::row(tw + xr * LD + rowq + 32 * ks);
          f32x4 m[4];
#pragma unroll
          for (int yt = 0; yt < 4; ++yt) m[yt] = zero4();
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int yt = 0; yt < 4; ++yt)
              m[yt] = X::mma(X::row(tz + (16 * yt + c) * LD + rowq + 32 * ks), qf[ks], m[yt]);
#pragma unroll
          for (int yt = 0; yt < 4; ++yt) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool in = yt < w || (yt == w && 4 * gq + j < c);
              const float x = in ? s_out * (m[yt][j] * p[yt][j]) : 0.f;
              r += x;
              const float cs = row16_sum_dpp(x);
              if (c == 0) csum[par][w][16 * yt + 4 * gq + j] = cs;
            }
          }
          r += __shfl_xor(r, 16, 64);
          r += __shfl_xor(r, 32, 64);
          if (gq == 0) rsum[par][xr] = r;
        }
      }
      const auto store_p = [&]() {
#pragma unroll
        for (int yt = 0; yt < 4; ++yt) {
          if (PT::kRev ? yt < (w & 2) : yt > (w | 1)) continue;
          E *const to = tp + (p_slot<PT::kRev>(w, yt) * kPTerms * 64 + lane) * 4;
          store4(to, p[yt]);
          if (kPTerms == 2) {
            f32x4 x = p[yt], unused = zero4();
            X::residual(X::round(x, unused), x, unused);
            store4(to + 256, x);
          }
        }
      };
      if (!PT::kDots) store_p();

      // the state's share: 32 rows of the state at a time, split once for the four row tiles
#pragma unroll
      for (int xt = 0; xt < 4; ++xt)
#pragma unroll
        for (int t = 0; t < NT; ++t) o[xt][t] = zero4();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        Frag sf[kStateTerms][NT], xf[4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          f32x4 s0 = S[2 * ks][t], s1 = S[2 * ks + 1][t];
#pragma unroll
          for (int i = 0; i < kStateTerms; ++i) {
            sf[i][t] = X::round(s0, s1);
            if (i + 1 < kStateTerms) X::residual(sf[i][t], s0, s1);
          }
        }
#pragma unroll
        for (int xt = 0; xt < 4; ++xt) {
          xf[xt] = X::row(tx + (16 * xt + c) * LD + rowq + 32 * ks);
        }
#pragma unroll
        for (int i = 0; i < kStateTerms; ++i)
#pragma unroll
          for (int xt = 0; xt < 4; ++xt)
#pragma unroll
            for (int t = 0; t < NT; ++t) o[xt][t] = X::mma(sf[i][t], xf[xt], o[xt][t]);
        sched_fence();
      }
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
            const f32x4 wv = load4(tw + xr * LD + X::place(c, out_col) + 4 * t);
#pragma unroll
            for (int j = 0; j < 4; ++j) d += wv[j] * o[xt][t][j];
          }
          d += __shfl_xor(d, 16, 64);
          d += __shfl_xor(d, 32, 64);
          if (gq == 0) dots[par][w][xr] = s_out * d;
        }
      }
      lds_barrier();
      if (PT::kDots) {
        store_p();
        lds_barrier();
      }
    }

    // z's columns of this wave: rows 32 kb + (order)
    Frag zf[2][NT];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        zf[kb][t] = X::template column<LD>(tz, 32 * kb, colq[t], col[t], c, gq);

    if constexpr (!PT::kSum) {
      const int64_t n_rows = t_end - t0;
#pragma unroll
      for (int xt = 0; xt < 4; ++xt) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          if (PT::kRev ? 2 * kb + 1 < xt : 2 * kb > xt) continue;
#pragma unroll
          for (int i = 0; i < kPTerms; ++i) {
            const Frag pf = X::pair(tp + ((p_slot<PT::kRev>(xt, 2 * kb) * kPTerms + i) * 64 + lane) * 4,
                                    kPTerms * 256);
#pragma unroll
            for (int t = 0; t < NT; ++t) o[xt][t] = X::mma(zf[kb][t], pf, o[xt][t]);
          }
        }
        const int xr = 16 * xt + c;
        if (xr < n_rows) {
          char *const base = static_cast<char *>(a.out) + ((t0 + 16 * xt) * out_heads + out_head) * D * out_size;
#pragma unroll
          for (int t = 0; t < NT; ++t) o[xt][t] *= s_out;
          if (PT::kDots && a.out_f32) {
            float *to = reinterpret_cast<float *>(base + v_out);
            if (NT == 2) store8(to, o[xt][0], o[xt][NT - 1]);
            else store4(to, o[xt][0]);
          } else {
            E *to = reinterpret_cast<E *>(base + v_out);
            if (NT == 2) store8(to, o[xt][0], o[xt][NT - 1]);
            else store4(to, o[xt][0]);
          }
        }
      }
    }

    sched_fence();
    if (PT::kDots && it + 1 < nsteps) fetch(ch + step);

    // the state after the chunk
    const float decay = sh_decay;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) S[m][t] *= decay;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const f32x4 fa = lds_f32x4(f_y + 32 * kb + 4 * gq), fb = lds_f32x4(f_y + 32 * kb + 16 + 4 * gq);
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
      for (int m = 0; m < MT; m += 2) {
        Frag yf[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          yf[i] = X::template column<LD>(ty, 32 * kb, 16 * (m + i) + 4 * (c & 3), 16 * (m + i) + c, c, gq);
        const auto add = [&](const Frag(&b)[NT]) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) S[m + i][t] = X::mma(yf[i], b[t], S[m + i][t]);
        };
        add(b1);
        if constexpr (kB) {
          add(b2);
          if (precise) add(b3);
        }
      }
      sched_fence();
    }
    if (w == kDecayWave && it + 1 < nsteps) make_decays();
  }
  if (PT::kDots && nsteps > 0) {
    __syncthreads();
    flush_dots(ch - step, (nsteps - 1) & 1);
  }

  const auto store_state = [&](float *to) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) to[(16 * m + 4 * gq + j) * D + col[t]] = S[m][t][j];
  };
  if (PT::kSum) {
    store_state((PT::kRev ? a.unit_r : a.unit_s) + uh * D * D);
    if (w == kDecayWave && lane == 0)
      a.unit_decay[(PT::kRev ? a.units * a.H : 0) + uh] = exp2_fast(total.hi + total.lo);
  }
  if ((PASS == kLinFwd || PASS == kLinDv) && edge_out && a.final_state)
    store_state(a.final_state + ((int64_t)seq * a.H + h) * D * D);
  if (PASS == kLinDq) {  // <state, its gradient> at the unit's end
    const float *ds = last ? (a.dht ? a.dht + ((int64_t)seq * a.H + h) * D * D : nullptr)
                           : a.unit_r + uh * D * D;
    double d = 0.0;
    if (ds) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const f32x4 x = *reinterpret_cast<const f32x4 *>(ds + col[t] * D + 16 * m + 4 * gq);
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
    if (tid == 0) a.unit_dot[uh] = dots[0][0][0] + dots[0][1][0] + dots[0][2][0] + dots[0][3][0];
  }
}

namespace {

// The states at the units' starts from the units' own sums, in place: along each sequence of more
// than one unit, S <- decay_u S + sum_u, written where unit u + 1's sum was.  rev: the gradients at
// the units' ends, from the last unit to the first.  One thread per four elements of a state; the
// loads run kAhead units ahead of the chain.
constexpr int kAhead = 4;
template <bool REV>
__global__ __launch_bounds__(256) void lin_scan_kernel(LinArgs a, int D) {
  const int seq = blockIdx.x, h = blockIdx.y;
  const int64_t e = ((int64_t)blockIdx.z * 256 + threadIdx.x) * 4, DD = (int64_t)D * D;
  const int32_t b0 = a.cu[seq], b1 = a.cu[seq + 1];
  if (b0 < 0 || b1 < b0 || b1 > a.T || e >= DD) return;
  const int nch = (b1 - b0 + kChunk - 1) / kChunk, nu = (nch + a.L - 1) / a.L;
  if (nu < 2) return;
  const int64_t u0 = a.seq_unit[seq];
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
  float d[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int s = min(j, steps - 1);
    b[j] = *reinterpret_cast<const f32x4 *>(st + us(s) * row);
    d[j] = dec[(int64_t)us(s) * a.H];
  }
  for (int s0 = 0; s0 < steps; s0 += kAhead) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int s = s0 + j;
      if (s < steps) {
        S = d[j] * S + b[j];
        if (s + kAhead < steps) {
          b[j] = *reinterpret_cast<const f32x4 *>(st + us(s + kAhead) * row);
          d[j] = dec[(int64_t)us(s + kAhead) * a.H];
        }
        *reinterpret_cast<f32x4 *>(st + us(s + 1) * row) = S;
      }
    }
  }
}

// dg_t = <dS_t, e^{g_t} S_{t-1}> from its parts: the pairs within the chunk on both sides of t,
// and the scan of q . dq and k . dk (the states' shares) from the unit's end, where
// <S, dS> is known: sum_{s >= t} (q_s . dq_s - k_s . dk_s) + <S, dS>_end.  The pairs' part has
// no cancelling terms; the scan's terms are of the size of dg near them, and it restarts at every
// unit's end.  One wave per (unit, head), from the unit's last chunk to its first.  A token whose
// decay is zero in fp32 has no gradient.
__global__ __launch_bounds__(256) void lin_dg_kernel(LinArgs a) {
  const int lane = threadIdx.x & 63, h = blockIdx.y * 4 + (threadIdx.x >> 6);
  if (h >= a.H) return;
  const int64_t uh = (int64_t)blockIdx.x * a.H + h;
  Unit un{};
  bool ok = find_unit(a.cu, a.N, a.T, a.L, blockIdx.x, false, lane, un);
  int64_t t_beg = 0, t_end = 0;
  if (ok) {
    t_beg = a.cu[un.seq], t_end = a.cu[un.seq + 1];
    ok = t_beg >= 0 && t_end >= t_beg && t_end <= a.T && un.c1 > un.c0;
  }
  double sum = 0.0;
  if (ok) {
    double b = (double)a.unit_dot[uh];
    const float gh = a.g_head ? a.g[h] : 0.f;
    struct Part {
      float q, k, p, g;
    };
    const auto fetch = [&](int ch) {
      const int64_t t = t_beg + (int64_t)ch * kChunk + lane;
      Part x{0.f, 0.f, 0.f, 0.f};
      if (t < t_end) {
        const int64_t i = t * a.H + h;
        x.q = a.dg_q[i], x.k = a.dg_k[i], x.p = a.dg_pairs[i];
        x.g = a.g_head ? gh : a.g[i];
      }
      return x;
    };
    Part next = fetch(un.c1 - 1);
    for (int ch = un.c1 - 1; ch >= un.c0; --ch) {
      const Part x = next;
      if (ch > un.c0) next = fetch(ch - 1);
      double s = (double)x.q - (double)x.k;  // sum over the lanes from this one on
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const double y = __shfl_down(s, off, 64);
        if (lane + off < 64) s += y;
      }
      const int64_t t = t_beg + (int64_t)ch * kChunk + lane;
      const F2 lg = log2_decay(x.g);
      const double dg = lg.hi <= kNoDecay ? 0.0 : (double)x.p + s + b;
      if (t < t_end) {
        if (!a.g_head) a.dg[t * a.H + h] = (float)dg;
        sum += dg;
      }
      b += __shfl(s, 0, 64);
    }
  }
  if (a.g_head) {
    sum = wave_sum_f64(sum);
    if (lane == 0) a.dg_unit[uh] = sum;
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

template <class E>
__global__ __launch_bounds__(256) void lin_group_sum_kernel(const float *__restrict__ part, int64_t n4,
                                                            int G, int D4, E *__restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
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

template <class E, int D, int PASS>
hipError_t launch_pass(const LinArgs &a, hipStream_t stream) {
  constexpr size_t lds = pass_lds_bytes<E, D, PASS>();
  if (lds > 65536) {  // above the default limit of dynamic LDS
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void *>(&lin_pass_kernel<E, D, PASS>),
        hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((lin_pass_kernel<E, D, PASS>), dim3((unsigned)a.units, a.H), dim3(256), lds,
                     stream, a);
  return hipGetLastError();
}

template <class E, int D>
hipError_t launch_pass_of(const LinArgs &a, LinPass pass, hipStream_t stream) {
  switch (pass) {
    case kLinFwd: return launch_pass<E, D, kLinFwd>(a, stream);
    case kLinDq: return launch_pass<E, D, kLinDq>(a, stream);
    case kLinDv: return launch_pass<E, D, kLinDv>(a, stream);
    case kLinDk: return launch_pass<E, D, kLinDk>(a, stream);
    case kLinSumFwd: return launch_pass<E, D, kLinSumFwd>(a, stream);
    default: return launch_pass<E, D, kLinSumRev>(a, stream);
  }
}

}  // namespace

hipError_t launch_linattn_pass(const LinArgs &a, int D, bool is_bf16, LinPass pass,
                               hipStream_t stream) {
  if (D == 128)
    return is_bf16 ? launch_pass_of<bf16, 128>(a, pass, stream)
                   : launch_pass_of<float, 128>(a, pass, stream);
  return is_bf16 ? launch_pass_of<bf16, 64>(a, pass, stream)
                 : launch_pass_of<float, 64>(a, pass, stream);
}

hipError_t launch_linattn_scan(const LinArgs &a, int D, bool rev, hipStream_t stream) {
  const dim3 grid((unsigned)a.N, a.H, D * D / 1024);
  if (rev) hipLaunchKernelGGL(lin_scan_kernel<true>, grid, dim3(256), 0, stream, a, D);
  else hipLaunchKernelGGL(lin_scan_kernel<false>, grid, dim3(256), 0, stream, a, D);
  return hipGetLastError();
}

hipError_t launch_linattn_dg(const LinArgs &a, hipStream_t stream) {
  hipLaunchKernelGGL(lin_dg_kernel, dim3((unsigned)a.units, (a.H + 3) / 4), dim3(256), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.g_head) return e;
  hipLaunchKernelGGL(lin_dg_head_kernel, dim3(a.H), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_linattn_group_sum(const float *part, int64_t T, int32_t H, int32_t HK, int32_t D,
                                    bool is_bf16, void *out, hipStream_t stream) {
  const int64_t n4 = T * HK * D / 4, blocks = std::min<int64_t>((n4 + 255) / 256, 16384);
  if (n4 <= 0) return hipSuccess;
  if (is_bf16)
    hipLaunchKernelGGL(lin_group_sum_kernel<bf16>, dim3((unsigned)blocks), dim3(256), 0, stream,
                       part, n4, H / HK, D / 4, static_cast<bf16 *>(out));
  else
    hipLaunchKernelGGL(lin_group_sum_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, stream,
                       part, n4, H / HK, D / 4, static_cast<float *>(out));
  return hipGetLastError();
}

hipError_t launch_linattn_zero(float *x, int64_t n, hipStream_t stream) {
  hipLaunchKernelGGL(lin_zero_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 1024)),
                     dim3(256), 0, stream, x, n);
  return hipGetLastError();
}

}  // namespace gdn
