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
template <>
struct Op<bf16> {
  typedef bf16x8 Frag;
  static constexpr int kPad = 8;
  static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) { return mma_bf16(a, b, c); }
  // a row: p at the row's first index plus 4 gq
  static __device__ __forceinline__ Frag row(const bf16 *p) {
    return cat8(lds_bf16x4(p), lds_bf16x4(p + 16));
  }
  // a column: rows row0 + (order) of column `col`; `colq` is the column this lane addresses
  template <int LD>
  static __device__ __forceinline__ Frag column(const bf16 *tile, int row0, int colq, int, int c,
                                                int gq) {
    const bf16 *p = tile + (row0 + 4 * gq + (c >> 2)) * LD + colq;
    return cat8(lds_tr16(p), lds_tr16(p + 16 * LD));
  }
  static __device__ __forceinline__ Frag round(f32x4 a, f32x4 b) { return to_bf16x8(a, b); }
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
  static __device__ __forceinline__ f32x4 lo_part(Frag f) { return f.a; }
  static __device__ __forceinline__ f32x4 hi_part(Frag f) { return f.b; }
};

// c + (a as a sum of TERMS rounded operands) . b, or with b the split one.
template <class E, int TERMS, bool SPLIT_A>
__device__ __forceinline__ f32x4 mma_split(f32x4 s0, f32x4 s1, typename Op<E>::Frag o, f32x4 c) {
  typedef Op<E> X;
#pragma unroll
  for (int i = 0; i < TERMS; ++i) {
    const typename X::Frag f = X::round(s0, s1);
    c = SPLIT_A ? X::mma(f, o, c) : X::mma(o, f, c);
    if (i + 1 < TERMS) {
      s0 -= X::lo_part(f);
      s1 -= X::hi_part(f);
    }
  }
  return c;
}

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

template <class E, int D, int PASS>
constexpr size_t pass_tile_bytes() {
  return (size_t)PassTraits<PASS>::kTiles * 64 * (D + Op<E>::kPad) * sizeof(E);
}

}  // namespace

template <class E, int D, int PASS>
__global__ __launch_bounds__(256) void lin_pass_kernel(LinArgs a) {
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
  constexpr int kPTerms = kB ? 2 : 1;

  extern __shared__ __attribute__((aligned(16))) char smem[];
  E *const ty = reinterpret_cast<E *>(smem);   // tiles [64][LD]: y, z, x, w
  E *const tz = ty + 64 * LD;
  E *const tx = tz + 64 * LD;
  E *const tw = tx + 64 * LD;
  __shared__ __attribute__((aligned(16))) float g_hi[64], g_lo[64], f_x[64], f_y[64];
  __shared__ float sh_decay;
  __shared__ float dots[4][64], rsum[64], csum[4][64];
  __shared__ int sh_unit[4];

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, c = lane & 15, gq = lane >> 4;
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
  const int seq = sh_unit[0], c0 = sh_unit[1], c1 = sh_unit[2];
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
  const void *px, *py, *pz, *pw = nullptr;
  int hx = h, hy = h, hz = h, hw = hk, nx = a.H, ny = a.H, nz = a.H;
  if (PASS == kLinFwd) {
    px = a.q, py = a.k, pz = a.v, hx = hy = hk, nx = ny = a.HK;
  } else if (PASS == kLinDq) {
    px = a.dout, py = a.v, pz = a.k, pw = a.q, hz = hk, nz = a.HK;
  } else if (PASS == kLinDv) {
    px = a.k, py = a.q, pz = a.dout, hx = hy = hk, nx = ny = a.HK;
  } else if (PASS == kLinDk) {
    px = a.v, py = a.dout, pz = a.q, pw = a.k, hz = hk, nz = a.HK;
  } else if (PASS == kLinSumFwd) {
    px = nullptr, py = a.k, pz = a.v, hy = hk, ny = a.HK;
  } else {
    px = nullptr, py = a.q, pz = a.dout, hy = hk, ny = a.HK;
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
  const int out_col = NT == 2 ? 32 * w + 8 * gq : 16 * w + 4 * gq;  // first column it stores

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
  const auto fetch = [&](int ch) {
    const int64_t t0 = t_beg + (int64_t)ch * kChunk;
    const int n = (int)(t_end - t0 < kChunk ? t_end - t0 : kChunk);
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      const int r = (tid + 256 * u) / UPR, o = (tid + 256 * u) % UPR * EPU;
      const uint4 z = {0u, 0u, 0u, 0u};
      sy[u] = sz[u] = sx[u] = sw[u] = z;
      if (r < n) {
        const int64_t t = t0 + r;
        sy[u] = *reinterpret_cast<const uint4 *>(static_cast<const E *>(py) + (t * ny + hy) * D + o);
        sz[u] = *reinterpret_cast<const uint4 *>(static_cast<const E *>(pz) + (t * nz + hz) * D + o);
        if (!PT::kSum)
          sx[u] = *reinterpret_cast<const uint4 *>(static_cast<const E *>(px) + (t * nx + hx) * D + o);
        if (PT::kDots)
          sw[u] = *reinterpret_cast<const uint4 *>(static_cast<const E *>(pw) +
                                                   (t * a.HK + hw) * D + o);
      }
    }
    if (w == 0) sg = lane < n ? a.g[a.g_head ? h : (t0 + lane) * a.H + h] : 0.f;
  };
  // dg's parts of the chunk before (every wave's share is in LDS)
  const auto flush_dots = [&](int ch) {
    if (!PT::kDots || w != 1) return;
    const int64_t t = t_beg + (int64_t)ch * kChunk + lane;
    float *const to = PASS == kLinDq ? a.dg_q : a.dg_k;
    const float d = dots[0][lane] + dots[1][lane] + dots[2][lane] + dots[3][lane];
    if (t < t_end) to[t * a.H + h] = d;
    if (PASS == kLinDq) {
      // sum over the pairs s >= t > i = sum_{s >= t} (row sum - column sum); rows from the end
      F2 x = F2{rsum[lane], 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j) x = add2(x, F2{-csum[j][lane], 0.f});
      const F2 up = wave_scan2(x);
      const float th = __shfl(up.hi, 63, 64), tl = __shfl(up.lo, 63, 64);
      const F2 rest = add2(add2(F2{th, tl}, F2{-up.hi, -up.lo}), x);
      if (t < t_end) a.dg_pairs[t * a.H + h] = rest.hi + rest.lo;
    }
  };

  F2 total{0.f, 0.f};  // kSum: the unit's whole log decay (wave 0)
  const int step = PT::kRev ? -1 : 1;
  int ch = PT::kRev ? c1 - 1 : c0;
  const int nsteps = c1 - c0;
  // terms of the state update: three where the state is written out or feeds dg
  const bool precise = kB && (PT::kSum || PT::kDots || (edge_out && a.final_state != nullptr));
  if (nsteps > 0) fetch(ch);
  for (int it = 0; it < nsteps; ++it, ch += step) {
    const int64_t t0 = t_beg + (int64_t)ch * kChunk;
    __syncthreads();
    if (it > 0) flush_dots(ch - step);
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      const int o = (tid + 256 * u) / UPR * LD + (tid + 256 * u) % UPR * EPU;
      *reinterpret_cast<uint4 *>(ty + o) = sy[u];
      *reinterpret_cast<uint4 *>(tz + o) = sz[u];
      if (!PT::kSum) *reinterpret_cast<uint4 *>(tx + o) = sx[u];
      if (PT::kDots) *reinterpret_cast<uint4 *>(tw + o) = sw[u];
    }
    if (w == 0) {
      const F2 G = wave_scan2(log2_decay(sg));
      const F2 GC = F2{__shfl(G.hi, 63, 64), __shfl(G.lo, 63, 64)};
      const float from_start = exp2_fast(G.hi + G.lo);
      const float to_end = exp2_fast((GC.hi - G.hi) + (GC.lo - G.lo));
      g_hi[lane] = G.hi;
      g_lo[lane] = G.lo;
      f_x[lane] = PT::kRev ? to_end : from_start;
      f_y[lane] = PT::kRev ? s_in * from_start : to_end;
      if (lane == 0) sh_decay = exp2_fast(GC.hi + GC.lo);
      total = add2(total, GC);
    }
    __syncthreads();
    if (it + 1 < nsteps) fetch(ch + step);

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
      for (int xt = 0; xt < 4; ++xt) {  // 16 output rows
        const int xr = 16 * xt + c;
        Frag xf[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) xf[ks] = X::row(tx + xr * LD + 32 * ks + 4 * gq);
        f32x4 o[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {  // the state's share
          o[t] = zero4();
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
            o[t] = mma_split<E, kStateTerms, true>(S[2 * ks][t], S[2 * ks + 1][t], xf[ks], o[t]);
          o[t] *= f_x[xr];
        }
        if (PT::kDots) {  // x's share of dg: w . (the state's share of the output)
          float d = 0.f;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const f32x4 wv = load4(tw + xr * LD + out_col + 4 * t);
#pragma unroll
            for (int j = 0; j < 4; ++j) d += wv[j] * o[t][j];
          }
          d += __shfl_xor(d, 16, 64);
          d += __shfl_xor(d, 32, 64);
          if (gq == 0) dots[w][xr] = s_out * d;
        }
        // the pairs within the chunk
        f32x4 p[4];
        const float xh = g_hi[xr], xl = g_lo[xr];
#pragma unroll
        for (int yt = 0; yt < 4; ++yt) {
          p[yt] = zero4();
          if (PT::kRev ? yt < xt : yt > xt) continue;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
            p[yt] = X::mma(X::row(ty + (16 * yt + c) * LD + 32 * ks + 4 * gq), xf[ks], p[yt]);
          const f32x4 yh = lds_f32x4(g_hi + 16 * yt + 4 * gq);
          const f32x4 yl = lds_f32x4(g_lo + 16 * yt + 4 * gq);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int yr = 16 * yt + 4 * gq + j;
            const float e = PT::kRev ? (yh[j] - xh) + (yl[j] - xl) : (xh - yh[j]) + (xl - yl[j]);
            const bool in = yt != xt || (PT::kRev ? yr >= xr : yr <= xr);
            p[yt][j] = in ? s_in * (p[yt][j] * exp2_fast(e)) : 0.f;
          }
        }
        if (PASS == kLinDq) {  // pairs strictly apart: (q . k) (do . v) decayed, by wave xt
          if (w == xt) {
            float r = 0.f;
            Frag qf[KS];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) qf[ks] = X::row(tw + xr * LD + 32 * ks + 4 * gq);
#pragma unroll
            for (int yt = 0; yt < 4; ++yt) {
              f32x4 m = zero4();
              if (yt <= xt) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                  m = X::mma(X::row(tz + (16 * yt + c) * LD + 32 * ks + 4 * gq), qf[ks], m);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const bool in = yt < xt || (yt == xt && 4 * gq + j < c);
                const float x = in ? s_out * (m[j] * p[yt][j]) : 0.f;
                r += x;
                const float cs = row16_sum_dpp(x);
                if (c == 0) csum[w][16 * yt + 4 * gq + j] = cs;
              }
            }
            r += __shfl_xor(r, 16, 64);
            r += __shfl_xor(r, 32, 64);
            if (gq == 0) rsum[xr] = r;
          }
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          if (PT::kRev ? 2 * kb + 1 < xt : 2 * kb > xt) continue;
#pragma unroll
          for (int t = 0; t < NT; ++t)
            o[t] = mma_split<E, kPTerms, false>(p[2 * kb], p[2 * kb + 1], zf[kb][t], o[t]);
        }
        if (xr < n_rows) {
          const int64_t row = (t0 + xr) * (PT::kGrad && PASS != kLinDv && !a.out_f32 ? a.HK : a.H) +
                              (PT::kGrad && PASS != kLinDv && !a.out_f32 ? hk : h);
#pragma unroll
          for (int t = 0; t < NT; ++t) o[t] *= s_out;
          if (PT::kDots && a.out_f32) {
            float *to = static_cast<float *>(a.out) + row * D + out_col;
            if (NT == 2) store8(to, o[0], o[NT - 1]);
            else store4(to, o[0]);
          } else {
            E *to = static_cast<E *>(a.out) + row * D + out_col;
            if (NT == 2) store8(to, o[0], o[NT - 1]);
            else store4(to, o[0]);
          }
        }
      }
    }

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
          u -= X::lo_part(b1[t]), v -= X::hi_part(b1[t]);
          b2[t] = X::round(u, v);
          u -= X::lo_part(b2[t]), v -= X::hi_part(b2[t]);
          b3[t] = X::round(u, v);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const Frag yf = X::template column<LD>(ty, 32 * kb, 16 * m + 4 * (c & 3), 16 * m + c, c, gq);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          S[m][t] = X::mma(yf, b1[t], S[m][t]);
          if constexpr (kB) {
            S[m][t] = X::mma(yf, b2[t], S[m][t]);
            if (precise) S[m][t] = X::mma(yf, b3[t], S[m][t]);
          }
        }
      }
    }
  }
  if (PT::kDots && nsteps > 0) {
    __syncthreads();
    flush_dots(ch - step);
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
    if (tid == 0) a.unit_decay[(PT::kRev ? a.units * a.H : 0) + uh] = exp2_fast(total.hi + total.lo);
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
    if (lane == 0) dots[w][0] = (float)d;
    __syncthreads();
    if (tid == 0) a.unit_dot[uh] = dots[0][0] + dots[1][0] + dots[2][0] + dots[3][0];
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
  constexpr size_t lds = pass_tile_bytes<E, D, PASS>();
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
