// Products of few rows with weights of 4 bits: y[t][n] = sum_k x[t][k] W[n][k],
// W[n][k] = e2m1(code) * 2^(byte - 127) with a byte for each 32 inputs.
//
// Packed weights.  A tile is 16 outputs (lane % 16) by 512 inputs; its 16
// blocks of 32 inputs are numbered 4 t + q, q = lane / 16.  Codes of a tile are
// [t][lane][16 bytes], its scales [lane][t]: one load of 1 KB a wave for a t, in
// the operand order of the matrix instructions, and one word a lane for the
// four scales.  A t is 128 adjacent inputs, so that a load of rows takes 64
// adjacent bytes of 8-bit rows, and two of 16-bit rows a whole line.  Outputs and inputs beyond the matrix have codes of 0.
#include <type_traits>

#include "common.h"
#include "launch.h"

namespace gdn {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int W4_TILE = 16 * 512 / 2;        // code bytes of a tile
__host__ __device__ inline int w4_ktiles(int k) { return (k + 511) / 512; }

// e8m0 as a float for the conversions, which read its exponent only: 0 is
// 2^-127, 255 NaN.
__device__ __forceinline__ float scale_f(uint32_t byte) {
  return __uint_as_float(byte << 23 | 0x00400000u);
}

// Eight codes as bf16 (exact: two significant bits).
__device__ __forceinline__ bf16x8 codes8(uint32_t w, float s) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <typename T>
__device__ __forceinline__ void put4(T* y, int64_t n, int64_t n_all, floatx4 v) {
  if (n + 4 <= n_all) {
    store4(y + n, v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < n_all) y[n + i] = from_f<T>(v[i]);
  }
}

// The same as fp16, exact for scales of 2^-13 to 2^13 (0.5 * 2^-13 is the
// smallest normal number); whether all four scales of a tile's lane are.
__device__ __forceinline__ fp16x8 codes8_f16(uint32_t w, float s) {
  typedef _Float16 fp16x2 __attribute__((ext_vector_type(2)));
  const auto a = __builtin_bit_cast(fp16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0));
  const auto b = __builtin_bit_cast(fp16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1));
  const auto c = __builtin_bit_cast(fp16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2));
  const auto d = __builtin_bit_cast(fp16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3));
  return fp16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ bool scales_f16(uint32_t sc) {
  bool in = true;
#pragma unroll
  for (int t = 0; t < 4; ++t) in &= (sc >> (8 * t) & 255) - 114u <= 26u;
  return in;
}

// Eight fp16 values as two terms of bf16 whose sum they are (11 bits in 8 + 8).
// What is not finite stays in the first.
__device__ __forceinline__ void split8(const bf16x8& bits, bf16x8 (&out)[2]) {
  const fp16x8 v = __builtin_bit_cast(fp16x8, bits);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    out[0][j] = (bf16)(float)v[j];
    const float hi = (float)out[0][j];
    out[1][j] = (bf16)(__builtin_isfinite(hi) ? (float)v[j] - hi : 0.f);
  }
}

struct Mx8 {};      // rows in e4m3 with a scale for each 32 columns

// Rows lie in LDS in steps of COLS inputs, 512 bytes of a row in memory: 8- and
// 16-bit ones as they are, fp32 as three planes of bf16 whose sum they are (24
// bits in 8 + 8 + 8), taken apart once, where they are put there (taken apart
// by every lane that multiplies them one row by 2560 x 6144 took 11.2 us, so
// 5.5).  Planes have no padding; the 16-byte pieces of row i are permuted by
// i % 16, so that 16 lanes that read one piece of 16 rows touch every bank once.
template <typename X> struct Step {
  static constexpr int E = sizeof(X), TERMS = E == 4 ? 3 : 1;
  static constexpr int COLS = 512 / E, TS = COLS / 128;      // inputs and t's of a step
  static constexpr int PP = COLS / 8;                        // pieces of a plane's row
  // Pieces of a row change places by its number with the bit pairs exchanged: a
  // 16-byte access is served for lanes 0-3, 12-15 and 20-27 together and so on,
  // which read pieces d and d + 4 of different rows (by the number itself each
  // group met half of the banks twice: 48 rows by 20480 x 8192, 3.9 M conflict
  // cycles, none so).
  __device__ __forceinline__ static int at(int row, int piece) {
    return row * PP + (piece ^ ((row >> 2 & 3) | (row & 3) << 2));
  }
  // piece i of row `row` in memory into planes `stride` pieces apart
  __device__ __forceinline__ static void put(uint4* planes, int stride, int row, int i, const uint4& raw) {
    if constexpr (TERMS == 1) {
      planes[at(row, i)] = raw;
    } else {
      // A term is the value's upper 16 bits (8 significant ones), cut, not
      // rounded, so that what is left is exact and no term overflows.  What is
      // not finite stays in the first term.  Bits below 2^-133, which no bf16 term
      // holds, are lost (only values below 2^-109 have such).
      const float* p = reinterpret_cast<const float*>(&raw);
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __builtin_canonicalizef(p[j]);
#pragma unroll
      for (int u = 0; u < TERMS; ++u) {
        uint32_t w[2];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const uint32_t a = __float_as_uint(v[j]), b = __float_as_uint(v[j + 1]);
          w[j / 2] = __builtin_amdgcn_perm(b, a, 0x07060302u);     // the upper halves
          const float c = v[j] - __uint_as_float(a & 0xffff0000u), d = v[j + 1] - __uint_as_float(b & 0xffff0000u);
          v[j] = c == c ? c : 0.f;               // an infinity leaves NaN
          v[j + 1] = d == d ? d : 0.f;
        }
        reinterpret_cast<uint2*>(planes + u * stride + at(row, i / 2))[i % 2] = make_uint2(w[0], w[1]);
      }
    }
  }
};
template <> struct Step<Mx8> {
  static constexpr int E = 1, TERMS = 1, COLS = 512, TS = 4, PP = 32;
  __device__ __forceinline__ static int at(int row, int piece) { return row * PP + (piece ^ (row & 15)); }
  __device__ __forceinline__ static void put(uint4* planes, int, int row, int i, const uint4& raw) {
    planes[at(row, i)] = raw;
  }
};

// What a lane reads of its row for 128 inputs, t of a step.
template <typename X> struct RowPart {
  bf16x8 b[Step<X>::TERMS][4];
  __device__ __forceinline__ void read(const uint4* planes, int stride, int row, int t, int q) {
#pragma unroll
    for (int u = 0; u < Step<X>::TERMS; ++u)
#pragma unroll
      for (int d = 0; d < 4; ++d)
        b[u][d] = __builtin_bit_cast(bf16x8, planes[u * stride + Step<X>::at(row, 4 * (4 * t + q) + d)]);
  }
};

// 8-bit rows go through the scaled instruction, which takes codes, values and
// scales as they are.  It adds the products of eight adjacent inputs with 13
// bits below the largest (measured: 256 + 2^-5 counts, 256 + 2^-6 does not,
// inputs eight apart add in full), 2^9 times finer than the rows' steps; all
// other sums are fp32.  Through bf16, which is exact, the same rows would cost
// four instructions of half the rate and sixteen conversions for its one.
template <> struct RowPart<Mx8> {
  // The instruction's 8-bit operand: lane group q holds columns 16 q .. 16 q +
  // 15 and 64 + 16 q .. of its 128, the scale of lane group q that of columns
  // 32 q .. 32 q + 31.
  uint4 lo, hi;
  int scale;
  __device__ __forceinline__ void read(const uint4* planes, int, int row, int t, int q) {
    lo = planes[Step<Mx8>::at(row, 8 * t + q)];
    hi = planes[Step<Mx8>::at(row, 8 * t + 4 + q)];
  }
};

template <int T>
__device__ __forceinline__ floatx4 mx_mma(const uint4& w, int sc, const RowPart<Mx8>& x, floatx4 acc) {
  const v8i av = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
  const v8i bv = {(int)x.lo.x, (int)x.lo.y, (int)x.lo.z, (int)x.lo.w,
                  (int)x.hi.x, (int)x.hi.y, (int)x.hi.z, (int)x.hi.w};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc, 4, 0, T, sc, 0, x.scale);
}

// acc[n][m] += the weights' tiles n by the rows' tiles m over 128 inputs.
// fp16 rows meet weights in fp16 (near: all scales are such that they are exact
// there) or else are taken apart into bf16: 9 rows by 2560 x 6144 take 4.6 us with
// the first and 7.9 with the second.
template <int T, typename X, int NT, int MT>
__device__ __forceinline__ void products(const uint4 (&w)[NT], const uint32_t (&sc)[NT], bool near,
                                         const RowPart<X> (&x)[MT], floatx4 (&acc)[NT][MT]) {
  if constexpr (__is_same(X, Mx8)) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[n][m] = mx_mma<T>(w[n], (int)sc[n], x[m], acc[n][m]);
    return;
  } else if (__is_same(X, fp16) && near) {
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t ws[4] = {w[n].x, w[n].y, w[n].z, w[n].w};
        const fp16x8 av = codes8_f16(ws[d], scale_f(sc[n] >> (8 * T) & 255));
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, __builtin_bit_cast(fp16x8, x[m].b[0][d]), acc[n][m],
                                                             0, 0, 0);
      }
  } else {
    constexpr int TERMS = __is_same(X, fp16) ? 2 : Step<X>::TERMS;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      bf16x8 b[MT][TERMS];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if constexpr (__is_same(X, fp16)) split8(x[m].b[0][d], b[m]);
        else
#pragma unroll
          for (int u = 0; u < TERMS; ++u) b[m][u] = x[m].b[u][d];
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t ws[4] = {w[n].x, w[n].y, w[n].z, w[n].w};
        const bf16x8 av = codes8(ws[d], scale_f(sc[n] >> (8 * T) & 255));
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int u = 0; u < TERMS; ++u)
            acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, b[m][u], acc[n][m], 0, 0, 0);
      }
    }
  }
}

// ---------------------------------------------------------------- few rows
// A tile of 16 outputs a workgroup, up to 2 RP rows.  Its waves share the
// inputs out, tile s of 512 to wave s % waves, and join their sums through LDS
// in wave order.  Every wave turns its inputs of the rows through LDS of its
// own: lanes read whole lines of a row, where an operand's own addresses are 64
// different ones (9 rows of bf16 by 2560 x 6144: 6.1 -> 4.4 us).  The weights are
// the A operand, so that a lane ends with four adjacent outputs of a row.
template <typename X, typename Y, int RP>
__global__ void __launch_bounds__(1024) w4_kernel(W4Args a) {
  constexpr bool MX = __is_same(X, Mx8);
  constexpr int E = Step<X>::E, TS = Step<X>::TS, PLANE = 2 * RP * Step<X>::PP,
                AHEAD = E == 2 && RP * __is_same(X, fp16) < 8 ? 2 : 1;     // steps asked for together (registers)
  extern __shared__ uint4 stage[];      // [wave][plane][2 RP rows], then the waves' sums
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int kt = w4_ktiles(a.k), rows = (int)a.rows;
  const int64_t tile0 = (int64_t)blockIdx.x * kt;
  const uint4* codes = (const uint4*)a.packed;
  const uint32_t* scales = (const uint32_t*)((const uint8_t*)a.packed + a.scales_at);
  uint4* mine = stage + wave * (Step<X>::TERMS * PLANE);
  const int piece = lane & 31, rr = r < 2 * RP ? r : 2 * RP - 1;
  const uint8_t* x[RP];                 // rows beyond the last read it; their sums are not stored
#pragma unroll
  for (int i = 0; i < RP; ++i) {
    const int row = 2 * i + (lane >> 5);
    x[i] = (const uint8_t*)a.x + (row < rows ? row : rows - 1) * a.ldx * E;
  }
  const uint8_t* xs = MX ? a.xs + (r < rows ? r : rows - 1) * a.ldxs : nullptr;
  floatx4 acc[1][1] = {{zero4()}};
  for (int s = wave; s < kt; s += waves) {
    uint4 w[4], raw[AHEAD][RP];
    const uint32_t sc = (scales + (tile0 + s) * 64)[lane];
#pragma unroll
    for (int t = 0; t < 4; ++t) w[t] = (codes + ((tile0 + s) * 4 + t) * 64)[lane];
    const bool near = __is_same(X, fp16) && __all(scales_f16(sc));
    int sx[4];
    if constexpr (MX)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int b = s * 16 + 4 * t + q;
        sx[t] = xs[b * 32 < a.k ? b : 0];
      }
#pragma unroll
    for (int h = 0; h < E; ++h) {
      if (h % AHEAD == 0)
#pragma unroll
        for (int g = 0; g < AHEAD; ++g) {
          const int at = (s * E + h + g) * 512 + piece * 16;
#pragma unroll
          for (int i = 0; i < RP; ++i) raw[g][i] = *(const uint4*)(x[i] + (at < a.k * E ? at : 0));
        }
      // inputs beyond the matrix become zero: their weights are, but what was read may not be finite
      const bool in = (s * E + h) * 512 + piece * 16 < a.k * E;
      wave_lds_order();
#pragma unroll
      for (int i = 0; i < RP; ++i)
        Step<X>::put(mine, PLANE, 2 * i + (lane >> 5), piece, in ? raw[h % AHEAD][i] : make_uint4(0, 0, 0, 0));
      wave_lds_order();
#define GDN_W4_PART(T)                                                                              \
  if constexpr (T < TS) {                                                                           \
    RowPart<X> part[1];                                                                             \
    part[0].read(mine, PLANE, rr, T, q);                                                            \
    if constexpr (MX) part[0].scale = (s * 16 + 4 * T + q) * 32 < a.k ? sx[T] : 127;                \
    const uint4 wt[1] = {w[MX ? T : h * TS + T]};                                                   \
    const uint32_t st[1] = {MX ? sc : sc >> (8 * (h * TS))};                                        \
    products<T, X, 1, 1>(wt, st, near, part, acc);                                                  \
  }
      GDN_W4_PART(0) GDN_W4_PART(1) GDN_W4_PART(2) GDN_W4_PART(3)
#undef GDN_W4_PART
    }
  }
  floatx4 v = acc[0][0];
  if (waves > 1) {
    __syncthreads();
    floatx4* sums = (floatx4*)stage;
    sums[wave * 64 + lane] = v;
    __syncthreads();
    if (wave > 0) return;
    for (int u = 1; u < waves; ++u) v += sums[u * 64 + lane];
  }
  if (r < rows) put4((Y*)a.y + r * a.ldy, (int64_t)blockIdx.x * 16 + 4 * q, a.n, v);
}

// ---------------------------------------------------------------- more rows
// Rows staged in LDS, where the waves of a workgroup share them: WN waves side
// by side take NT tiles of 16 outputs each, WK such groups share the inputs
// out.  A step is 512 bytes of each of 16 MT rows; while it is multiplied the
// next one's rows and weights are on their way.
template <typename X, int MT> struct StageLds {
  uint4 x[2][Step<X>::TERMS * 16 * MT * Step<X>::PP];
  uint32_t xs[__is_same(X, Mx8) ? 2 : 1][__is_same(X, Mx8) ? 16 * MT * 4 : 1];
};

template <typename X, typename Y, int WN, int WK, int NT, int MT>
__global__ void __launch_bounds__(64 * WN * WK) w4_rows_kernel(W4Args a) {
  typedef Step<X> S;
  constexpr bool MX = __is_same(X, Mx8);
  constexpr int GT = 64 * WN, NL = 16 * MT * 32 / GT, NS = (16 * MT * 4 + GT - 1) / GT;
  __shared__ union {
    StageLds<X, MT> st[WK];
    floatx4 part[WK > 1 ? (WK - 1) * WN * NT * MT * 64 : 1];
  } lds;
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wn = wave % WN, g = wave / WN;
  const int gt = threadIdx.x % GT;
  StageLds<X, MT>& st = lds.st[g];
  const int kt = w4_ktiles(a.k), tiles = (a.n + 15) / 16;
  const int steps_all = (a.k * S::E + 511) / 512;      // of 512 bytes of a row
  const int steps = (steps_all + WK - 1) / WK;         // a group's, the last one's perhaps empty
  // Workgroups go to the eight XCDs in turn.  Those of one piece of outputs and
  // all pieces of rows follow each other on one of them, so that its L2 serves
  // the weights but once (16480 x 2560, 64 8-bit rows in 32s: 11.6 -> 9.4 us).
  const int64_t turn = blockIdx.x / 8, block = turn / a.row_blocks * 8 + blockIdx.x % 8;
  const int n0 = (int)((block * WN + wn) * NT);
  if (block * WN * NT >= tiles) return;       // the whole workgroup
  const uint4* codes = (const uint4*)a.packed + lane;
  const uint32_t* scales = (const uint32_t*)((const uint8_t*)a.packed + a.scales_at) + lane;

  for (int64_t m0 = turn % a.row_blocks * 16 * MT; m0 < a.rows; m0 += a.row_blocks * 16 * MT) {
    const uint8_t* xrow[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int64_t m = m0 + (gt + GT * i) / 32;
      xrow[i] = (const uint8_t*)a.x + (m < a.rows ? m : a.rows - 1) * a.ldx * S::E;
    }
    uint4 xn[NL], wn_[S::TS][NT];
    uint32_t sn[NT], xsn[MX ? NS : 1];
    const auto ask = [&](int j) {      // the group's step j
      const int step = j * WK + g, t0 = step * S::TS;  // t's of the whole row
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int64_t tile = (int64_t)(n0 + n < tiles ? n0 + n : tiles - 1) * kt + (t0 / 4 < kt ? t0 / 4 : kt - 1);
        sn[n] = scales[tile * 64];
#pragma unroll
        for (int t = 0; t < S::TS; ++t) wn_[t][n] = codes[(tile * 4 + t0 % 4 + t) * 64];
      }
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int at = step * 512 + (gt + GT * i) % 32 * 16;
        xn[i] = *(const uint4*)(xrow[i] + (at < a.k * S::E ? at : 0));
        if (at >= a.k * S::E) xn[i] = make_uint4(0, 0, 0, 0);
      }
      if constexpr (MX) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const int id = gt + GT * i, b = step * 16 + id % 4 * 4, all = a.k / 32;
          const int64_t m = m0 + id / 4;
          xsn[i] = 0x7f7f7f7f;
          if (id < 16 * MT * 4) {
            const uint8_t* p = a.xs + (m < a.rows ? m : a.rows - 1) * a.ldxs + b;
            if (b + 4 <= all) {
              __builtin_memcpy(&xsn[i], p, 4);
            } else {
              for (int u = 0; u < 4; ++u)
                if (b + u < all) xsn[i] = (xsn[i] & ~(255u << (8 * u))) | (uint32_t)p[u] << (8 * u);
            }
          }
        }
      }
    };
    const auto keep = [&](int buf) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int id = gt + GT * i, row = id / 32;
        S::put(st.x[buf], 16 * MT * S::PP, row, id % 32, xn[i]);
      }
      if constexpr (MX) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
          if (gt + GT * i < 16 * MT * 4) st.xs[buf][gt + GT * i] = xsn[i];
      }
    };
    floatx4 acc[NT][MT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[n][m] = zero4();
    ask(0);
    keep(0);
    __syncthreads();
    for (int j = 0; j < steps; ++j) {
      uint4 w[S::TS][NT];
      uint32_t sc[NT];
      bool near = __is_same(X, fp16);
#pragma unroll
      for (int n = 0; n < NT; ++n) near = near && __all(scales_f16(sn[n]));
      const bool full = j * WK + g < steps_all;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        sc[n] = sn[n] >> (j * WK + g) * S::TS % 4 * 8;
#pragma unroll
        for (int t = 0; t < S::TS; ++t) w[t][n] = wn_[t][n];
      }
      if (j + 1 < steps) ask(j + 1);
      if (full) {
        const uint4* xb = st.x[j & 1];
#define GDN_W4_PART(T)                                                                                       \
  if constexpr (T < S::TS) {                                                                                 \
    RowPart<X> x[MT];                                                                                        \
    _Pragma("unroll") for (int m = 0; m < MT; ++m) {                                                         \
      x[m].read(xb, 16 * MT * S::PP, 16 * m + r, T, q);                                                      \
      if constexpr (MX) x[m].scale = (int)(st.xs[j & 1][(16 * m + r) * 4 + T] >> (8 * q));                   \
    }                                                                                                        \
    products<T, X, NT, MT>(w[T < S::TS ? T : 0], sc, near, x, acc);                                          \
  }
        GDN_W4_PART(0) GDN_W4_PART(1) GDN_W4_PART(2) GDN_W4_PART(3)
#undef GDN_W4_PART
      }
      if (j + 1 < steps) keep((j + 1) & 1);
      __syncthreads();
    }
    if constexpr (WK > 1) {            // the groups' sums, in group order
      if (g > 0)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            lds.part[((((g - 1) * WN + wn) * NT + n) * MT + m) * 64 + lane] = acc[n][m];
      __syncthreads();
      if (g == 0)
#pragma unroll
        for (int u = 0; u < WK - 1; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[n][m] += lds.part[(((u * WN + wn) * NT + n) * MT + m) * 64 + lane];
      __syncthreads();
    }
    if (g == 0)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int64_t row = m0 + 16 * m + r;
          if (row < a.rows) put4((Y*)a.y + row * a.ldy, (int64_t)(n0 + n) * 16 + 4 * q, a.n, acc[n][m]);
        }
  }
}

// ---------------------------------------------------------------- packing
// One wave a t of a tile: a lane takes block 4 t + q of its output.
//
// Of the smallest scale u that keeps a block within 6 = 0.75 * 2^3 and u / 2,
// which cuts its largest to 6, the one with the smaller squared error.  With
// y = w / (u / 2), A and B the nearest values of w under u and u / 2 in units
// of u / 2, the errors' difference is
//   sum (y - B)^2 - (y - A)^2 = sum (A - B) (2 y - (A + B)),
// one sum, most of whose terms are zero.  Near ties must not hang on the sum's
// order: of 16-bit weights it is exact in fp32 (where A and B differ, y is above
// 1/4, so that a term is a multiple of 2^-12; |A - B| and |2 y - (A + B)| are at
// most 8 each, 32 terms at most 2^11: 23 bits), of fp32 ones it is 64 bits.
typedef float floatx2 __attribute__((ext_vector_type(2)));
template <typename T>
__global__ void __launch_bounds__(256) w4_pack_kernel(const T* w, int64_t ldw, int n, int k, int64_t parts,
                                                      uint8_t* packed, int64_t scales_at) {
  constexpr int V = 16 / sizeof(T), P = 128 / V;       // values of a 16-byte piece, pieces of a row
  __shared__ uint4 turn[4][16 * (P + 1)];              // rows a piece apart: all banks once
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, r = lane & 15;
  const int kt = w4_ktiles(k);
  const int64_t part = (int64_t)blockIdx.x * 4 + wave, tile = part >> 2;
  const int t = (int)(part & 3);
  const int64_t row = tile / kt * 16 + r;
  const int k0 = (int)(tile % kt) * 512 + 128 * t + 32 * q;
  if (part < parts) {
#pragma unroll
    for (int i = 0; i < 16 * P / 64; ++i) {            // 16 lanes read 256 adjacent bytes of an output
      const int id = i * 64 + lane, piece = id % P;
      const int64_t at = tile / kt * 16 + id / P;
      const int c = (int)(tile % kt) * 512 + 128 * t + piece * V;
      turn[wave][id / P * (P + 1) + piece] = __builtin_bit_cast(
          uint4, __builtin_nontemporal_load(reinterpret_cast<const nt_u32x4*>(w + (at < n ? at : n - 1) * ldw + (c < k ? c : 0))));
    }
  }
  __syncthreads();
  if (part >= parts) return;
  uint32_t code[4] = {0, 0, 0, 0};
  int e = 0;             // of zeros, and beyond the matrix: products in fp16 want scales near 1
  if (row < n && k0 < k) {
    Raw8<T> raw[4];
    f8 v[4];
    uint32_t top = 0;                  // the largest magnitude's bits as a float; above those of infinity: NaN
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
        raw[d].v[i] = turn[wave][r * (P + 1) + q * (P / 4) + d * (P / 16) + i];
    if constexpr (sizeof(T) == 2) {
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      u16x2 most = {0, 0};
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t ws[4] = {raw[d].v[0].x, raw[d].v[0].y, raw[d].v[0].z, raw[d].v[0].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, ws[j] & 0x7fff7fffu));
      }
      const uint16_t one = most[0] > most[1] ? most[0] : most[1];
      top = __float_as_uint(to_f(__builtin_bit_cast(T, one)));
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      v[d] = raw_f8(raw[d]);
      if constexpr (sizeof(T) == 4)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t b = __float_as_uint(v[d].v[j]) & 0x7fffffffu;
          top = top > b ? top : b;
        }
    }
    if (top >= 0x7f800000u) {
      e = 128;
    } else if (top != 0) {
      const float amax = __uint_as_float(top);
      e = __builtin_amdgcn_frexp_expf(amax) - 3 + (__builtin_amdgcn_frexp_mantf(amax) > 0.75f);
      e = e < -127 ? -127 : e > 125 ? 125 : e;       // 6 * 2^125 is finite, 4 * 2^126 is not
      const float u = scale_f(e + 127), half = scale_f(e > -127 ? e + 126 : 0);
      uint32_t fine[4];
      typename std::conditional<sizeof(T) == 4, double, float>::type sum = 0;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        uint32_t cw = 0, cf = 0;
#define GDN_PAIR(I)                                                                                     \
  cw = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(cw, v[d].v[2 * I], v[d].v[2 * I + 1], u, I);            \
  cf = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(cf, v[d].v[2 * I], v[d].v[2 * I + 1], half, I);
        GDN_PAIR(0) GDN_PAIR(1) GDN_PAIR(2) GDN_PAIR(3)
#undef GDN_PAIR
#define GDN_PAIR(I)                                                                                     \
  {                                                                                                     \
    const floatx2 A = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw, 2.f, I);                             \
    const floatx2 B = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cf, 1.f, I);                             \
    _Pragma("unroll") for (int j = 0; j < 2; ++j)                                                       \
        sum += (A[j] - B[j]) * (ldexpf(v[d].v[2 * I + j], 2 - e) - (A[j] + B[j]));                      \
  }
        GDN_PAIR(0) GDN_PAIR(1) GDN_PAIR(2) GDN_PAIR(3)
#undef GDN_PAIR
        code[d] = cw;
        fine[d] = cf;
      }
      if (e > -127 && sum < 0) {
        --e;
#pragma unroll
        for (int d = 0; d < 4; ++d) code[d] = fine[d];
      }
    }
  }
  ((uint4*)packed)[part * 64 + lane] = make_uint4(code[0], code[1], code[2], code[3]);
  packed[scales_at + (tile * 64 + lane) * 4 + t] = (uint8_t)(e + 127);
}

// Codes [n][k/2] and scales [n][k/32] into the packed order.
__global__ void __launch_bounds__(256) w4_arrange_kernel(const uint8_t* codes, int64_t ldc, const uint8_t* scales,
                                                         int64_t lds, int n, int k, int64_t tiles, uint8_t* packed,
                                                         int64_t scales_at) {
  const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int kt = w4_ktiles(k);
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (tile >= tiles) return;
  const int64_t row = tile / kt * 16 + r;
  const int k0 = (int)(tile % kt) * 512 + q * 32;
  uint32_t sc = 0x7f7f7f7f;          // 1 beyond the matrix
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    uint4 c = make_uint4(0, 0, 0, 0);
    if (row < n && k0 + 128 * t < k) {
      c = *(const uint4*)(codes + row * ldc + (k0 + 128 * t) / 2);
      sc = (sc & ~(255u << (8 * t))) | (uint32_t)scales[row * lds + (k0 + 128 * t) / 32] << (8 * t);
    }
    ((uint4*)packed)[(tile * 4 + t) * 64 + lane] = c;
  }
  ((uint32_t*)(packed + scales_at))[tile * 64 + lane] = sc;
}

// Packed weights into dense rows of a storage type: one wave a t of a tile,
// turned in LDS so that 16 lanes store 256 adjacent bytes of an output.
template <typename T>
__global__ void __launch_bounds__(256) w4_unpack_kernel(const uint8_t* packed, int64_t scales_at, int n, int k,
                                                        int64_t parts, T* w, int64_t ldw) {
  constexpr int V = 16 / sizeof(T), P = 128 / V;       // values of a 16-byte piece, pieces of a row
  __shared__ uint4 turn[4][16 * (P + 1)];              // rows a piece apart: all banks once
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, r = lane & 15;
  const int kt = w4_ktiles(k);
  const int64_t part = (int64_t)blockIdx.x * 4 + wave, tile = part >> 2;
  const int t = (int)(part & 3);
  if (part < parts) {
    const uint4 c = ((const uint4*)packed)[part * 64 + lane];
    const uint32_t cs[4] = {c.x, c.y, c.z, c.w};
    const float s = scale_f(packed[scales_at + (tile * 64 + lane) * 4 + t]);
    uint4* at = turn[wave] + r * (P + 1) + q * (P / 4);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if constexpr (sizeof(T) == 4) {
#define GDN_PAIR(I) const floatx2 v##I = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cs[d], s, I);
        GDN_PAIR(0) GDN_PAIR(1) GDN_PAIR(2) GDN_PAIR(3)
#undef GDN_PAIR
        at[2 * d] = __builtin_bit_cast(uint4, floatx4{v0[0], v0[1], v1[0], v1[1]});
        at[2 * d + 1] = __builtin_bit_cast(uint4, floatx4{v2[0], v2[1], v3[0], v3[1]});
      } else if constexpr (__is_same(T, bf16)) {
        at[d] = __builtin_bit_cast(uint4, codes8(cs[d], s));
      } else {
#define GDN_PAIR(I) __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(cs[d], s, I))
        at[d] = make_uint4(GDN_PAIR(0), GDN_PAIR(1), GDN_PAIR(2), GDN_PAIR(3));
#undef GDN_PAIR
      }
    }
  }
  __syncthreads();
  if (part >= parts) return;
  const int64_t row0 = tile / kt * 16;
  const int k0 = (int)(tile % kt) * 512 + 128 * t;
#pragma unroll
  for (int i = 0; i < 16 * P / 64; ++i) {
    const int id = i * 64 + lane, row = id / P, piece = id % P;
    if (row0 + row < n && k0 + piece * V < k)
      store16_nt(w + (row0 + row) * ldw + k0 + piece * V, turn[wave][row * (P + 1) + piece]);
  }
}

static int64_t w4_tiles(int n, int k) { return (int64_t)((n + 15) / 16) * w4_ktiles(k); }
size_t w4_bytes(int n, int k) { return (size_t)w4_tiles(n, k) * (W4_TILE + 256); }
int64_t w4_scales_at(int n, int k) { return w4_tiles(n, k) * W4_TILE; }

template <typename X, typename Y, int RP> static hipError_t w4_go(const W4Args& a, hipStream_t st) {
  constexpr int LDS = 16 * 2 * RP * Step<X>::PP * Step<X>::TERMS, MOST = 160 * 1024 / LDS < 16 ? 160 * 1024 / LDS : 16;
  const int kt = w4_ktiles(a.k), turns = (kt + MOST - 1) / MOST, waves = (kt + turns - 1) / turns;
  hipLaunchKernelGGL((w4_kernel<X, Y, RP>), dim3((unsigned)((a.n + 15) / 16)), dim3(64 * waves), LDS * waves, st, a);
  return hipGetLastError();
}

template <typename X, typename Y, int WN, int WK, int NT, int MT>
static hipError_t w4_rows_go(const W4Args& args, hipStream_t st) {
  W4Args a = args;
  const int64_t mb = (a.rows + 16 * MT - 1) / (16 * MT), nb = (((a.n + 15) / 16 + NT * WN - 1) / (NT * WN) + 7) / 8 * 8;
  const int64_t most = ((int64_t)1 << 31) / (nb * 64 * WN * WK);
  a.row_blocks = mb < most ? mb : most < 1 ? 1 : most;
  hipLaunchKernelGGL((w4_rows_kernel<X, Y, WN, WK, NT, MT>), dim3((unsigned)(nb * a.row_blocks)), dim3(64 * WN * WK), 0,
                     st, a);
  return hipGetLastError();
}

// A unit is a tile of 16 outputs by one of 16 rows.  The inputs are shared out
// over as many waves a unit as leave all waves on the chip at once (about 16 a
// CU, 12 with 8-bit rows); beyond that, workgroups take 32 rows or more.  Fewer waves
// a unit leave CUs idle, more wait for a second round.  Measured, us a launch
// (outputs x inputs, rows: units; each with 4, 2 and 1 waves a unit, and with
// 1 and 32 rows):
//   bf16   2560 x 8192,  32:  320   9.4  14.0  19.6  25.9
//         10240 x 8192,  16:  640  13.8  16.2  21.2
//         10240 x 2560,  16:  640   7.1   6.6   8.1
//         10240 x 8192,  48: 1920  23.6  18.4  21.8  31.3
//         16480 x 2560,  48: 3090  18.5  13.0  11.3  13.9
//         20480 x 8192,  64: 5120  55.8  48.3  48.8  40.8
//   8 bit  2560 x 8192,  32:  320   6.4   9.2  11.4  14.1
//         10240 x 8192,  48: 1920  21.9  12.8  13.4  17.2
//         10240 x 2560,  48: 1920  15.4   6.9   6.0   7.3
//         16480 x 2560,  64: 4120  31.4  14.4  10.1   9.4
// Many rows (as prompts have them): two tiles of outputs a wave and 32 to 64
// rows, since a wave's reads of the rows from LDS and its conversions of the
// weights then serve more products.  1 tile by 32 rows, 2 by 32, 48 and 64:
//   bf16   2560 x 6144, 1024:10240  60.0  44.1  64.4  49.3
//         10240 x 2560,  192: 7680  16.5  16.5  19.4  17.9
//         20480 x 8192,  128:10240  63.9  57.6  53.8  66.8
//         16480 x 2560,  256:16480  31.5  30.9  33.7  34.4
//         20480 x 8192, 1024:81920   701   374   349   306 (1.1 PFLOP/s)
//   8 bit 10240 x 2560,  128: 5120   9.8  10.0   9.7  11.2
//         16480 x 2560,  128: 8240  14.1  14.2  12.4  19.6
//         20480 x 8192,  256:20480  71.6  63.6  58.1  87.3
//         20480 x 8192, 1024:81920   360   269   201   298
// (each on one set of values, pass after pass; the largest depend on the values and
// on the card's clock: under the profiler, random codes in three sets, 1024 rows
// by 20480 x 8192 take 348 to 406 us, 324 at best, and 8-bit rows 221 to 259.)
//
// fp16 rows of such calls take longer than bf16 ones (1024 rows by 20480 x 8192 538
// us against 348, by 2560 x 6144 62 against 50), fp32 rows, three terms, 2.4 to
// 3 times as long (1054 and 119).
//
// Few rows: every wave its own inputs, all of the weights asked for at once;
// against the above, of which one row takes as long as 16:
//   bf16   2560 x  6144:  1, 4, 8, 12, 16 rows  3.5  3.7  4.0  4.5  5.0    7.6
//          8192 x  4096:                        5.3  5.3  5.2  6.1  6.7    6.7
//         16480 x  2560:                        6.0  6.1  6.8  9.7 10.6    7.3
//         20480 x  8192:                       15.7 16.1 21.9 26.7 29.9   21.3
//   8 bit  2560 x  6144:                        2.9  3.3  4.0  4.6  5.1    5.1
//          8192 x  4096:                        4.8  4.9  5.7  6.2  6.8    5.5
//         16480 x  2560:                        5.3  5.5  5.8  7.0  9.1    6.5
//         20480 x  8192:                       14.7 14.5 21.1 26.8 30.1   19.9
template <typename X, typename Y> static hipError_t w4_m(const W4Args& a, hipStream_t st) {
  constexpr bool MX = __is_same(X, Mx8);
  const int64_t tiles = (a.n + 15) / 16, units = tiles * ((a.rows + 15) / 16);
  const bool deep = a.k >= 4096;
  if (a.rows <= 2) return w4_go<X, Y, 1>(a, st);
  if (a.rows <= 4) return w4_go<X, Y, 2>(a, st);
  if (a.rows <= 8 && (tiles <= 512 || !deep)) return w4_go<X, Y, 4>(a, st);
  if (a.rows <= 16 && tiles <= (MX ? 256 : 512)) return a.rows <= 12 ? w4_go<X, Y, 6>(a, st) : w4_go<X, Y, 8>(a, st);
  if (units <= 512 || (!MX && units <= 1024 && deep)) return w4_rows_go<X, Y, 2, 4, 1, 1>(a, st);
  if (units <= 1024 || (units <= 2048 && (!MX || deep))) return w4_rows_go<X, Y, 4, 2, 1, 1>(a, st);
  if (units <= 4096) return w4_rows_go<X, Y, 4, 1, 1, 1>(a, st);
  if (units <= 8192) return w4_rows_go<X, Y, 4, 1, 1, 2>(a, st);
  if (MX) return w4_rows_go<X, Y, 4, 1, 2, 3>(a, st);
  // 64 rows in three terms do not fit into LDS
  if (units <= 32768 || __is_same(X, float)) return w4_rows_go<X, Y, 4, 1, 2, 2>(a, st);
  return w4_rows_go<X, Y, 4, 1, 2, sizeof(X) == 2 ? 4 : 2>(a, st);
}

hipError_t launch_w4(const W4Args& a, gdn_dtype dt, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (a.xs)
    return dt == GDN_BF16 ? w4_m<Mx8, bf16>(a, st) : dt == GDN_FP16 ? w4_m<Mx8, fp16>(a, st) : w4_m<Mx8, float>(a, st);
  return dt == GDN_BF16 ? w4_m<bf16, bf16>(a, st) : dt == GDN_FP16 ? w4_m<fp16, fp16>(a, st) : w4_m<float, float>(a, st);
}

hipError_t launch_w4_pack(gdn_dtype dt, const void* w, int64_t ldw, int n, int k, void* packed, hipStream_t st) {
  const int64_t parts = 4 * w4_tiles(n, k), at = w4_scales_at(n, k);
  const dim3 grid((unsigned)((parts + 3) / 4));
  if (dt == GDN_BF16)
    hipLaunchKernelGGL(w4_pack_kernel<bf16>, grid, dim3(256), 0, st, (const bf16*)w, ldw, n, k, parts, (uint8_t*)packed, at);
  else if (dt == GDN_FP16)
    hipLaunchKernelGGL(w4_pack_kernel<fp16>, grid, dim3(256), 0, st, (const fp16*)w, ldw, n, k, parts, (uint8_t*)packed, at);
  else
    hipLaunchKernelGGL(w4_pack_kernel<float>, grid, dim3(256), 0, st, (const float*)w, ldw, n, k, parts, (uint8_t*)packed, at);
  return hipGetLastError();
}

hipError_t launch_w4_arrange(const void* codes, int64_t ldc, const void* scales, int64_t lds, int n, int k,
                             void* packed, hipStream_t st) {
  const int64_t tiles = w4_tiles(n, k);
  hipLaunchKernelGGL(w4_arrange_kernel, dim3((unsigned)((tiles + 3) / 4)), dim3(256), 0, st, (const uint8_t*)codes, ldc,
                     (const uint8_t*)scales, lds, n, k, tiles, (uint8_t*)packed, w4_scales_at(n, k));
  return hipGetLastError();
}

hipError_t launch_w4_unpack(gdn_dtype dt, const void* packed, int n, int k, void* w, int64_t ldw, hipStream_t st) {
  const int64_t parts = 4 * w4_tiles(n, k), at = w4_scales_at(n, k);
  const dim3 grid((unsigned)((parts + 3) / 4));
  if (dt == GDN_BF16)
    hipLaunchKernelGGL(w4_unpack_kernel<bf16>, grid, dim3(256), 0, st, (const uint8_t*)packed, at, n, k, parts, (bf16*)w, ldw);
  else if (dt == GDN_FP16)
    hipLaunchKernelGGL(w4_unpack_kernel<fp16>, grid, dim3(256), 0, st, (const uint8_t*)packed, at, n, k, parts, (fp16*)w, ldw);
  else
    hipLaunchKernelGGL(w4_unpack_kernel<float>, grid, dim3(256), 0, st, (const uint8_t*)packed, at, n, k, parts, (float*)w, ldw);
  return hipGetLastError();
}

}  // namespace gdn
