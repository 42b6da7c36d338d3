// The residual's addition with the zero-centred RMSNorm that follows it:
//   h = x + res,  y = h * rho * (1 + w),  rho = (mean h^2 + eps)^(-1/2)
// and its backward.  HBM-bound: each row is read once, held in registers and
// written once.  The norm reads the sum before h is rounded to its storage
// type, so y carries one rounding.
//
// A thread owns 8 columns (16 beyond 8192) for the whole call, with
// their weights in registers, and takes RB rows at a time, so that the loads
// of RB rows are on their way together (PF: the next rows' while these are
// worked on).  A row is owned by LPR lanes, or by all
// waves of a workgroup where it is wider than a wave's 512 columns.  Which
// products and sums are fused is written out, so that a row's result does not
// hang on the variant that a call's number of rows selects.
#include "common.h"
#include "launch.h"

namespace gdn {

// Sums of N values over a row's threads; every thread gets them.  red: two
// buffers used in turn, so that one barrier a call is enough.
template <int LPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[N], int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int m = LPR / 2; m >= 1; m >>= 1) v[i] += __shfl_xor(v[i], m);
  if (LPR == 64 && waves > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[wave][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int u = 0; u < waves; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += red[u][i];
  }
}

// e4m3 under the smallest power of two that keeps a group's largest within
// 448 = 0.875 * 2^9.  NaN stays NaN and leaves the scale to the others;
// infinities become NaN.
__device__ __forceinline__ int mx8_exponent(float amax) {
  int e = __builtin_amdgcn_frexp_expf(amax) - 9 + (__builtin_amdgcn_frexp_mantf(amax) > 0.875f);
  if (amax == 0.f) e = -127;
  if (__builtin_isinf(amax)) e = 127;
  return e < -127 ? -127 : e > 127 ? 127 : e;
}
__device__ __forceinline__ float amax4(const float* v) {
  return fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
}
__device__ __forceinline__ uint32_t mx8_word(const float* v, int e) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(v[0], -e), ldexpf(v[1], -e), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(v[2], -e), ldexpf(v[3], -e), lo, true);
}

// A thread's columns of piece p.  Where all tensors are 16-bit: 8 adjacent
// ones, a 16-byte access.  Where one is fp32: two runs of 4, as far apart as
// the row's threads reach, so that an access of 16 bytes a lane leaves no gaps
// between lanes; with 8 adjacent columns each access would touch every other
// 16 bytes (32768 x 2560 in
// fp32: 250 us, in runs 218; backward 281 and 235).
struct Cols {
  int a, b;
  bool in_a, in_b;       // columns that are not in the row read its first ones and count for nothing
};
template <bool SPLIT, int P> __device__ __forceinline__ void cols(Cols (&at)[P], int i, int threads, int n) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int a = SPLIT ? (2 * p * threads + i) * 4 : (p * threads + i) * 8;
    const int b = SPLIT ? a + threads * 4 : a + 4;
    at[p].in_a = a < n;
    at[p].in_b = b < n;
    at[p].a = at[p].in_a ? a : 0;
    at[p].b = at[p].in_b ? b : SPLIT ? 0 : 4;
  }
}

template <typename V, bool NT> __device__ __forceinline__ V ask(const void* p) {
  if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
  else return *reinterpret_cast<const V*>(p);
}
template <typename V, bool NT> __device__ __forceinline__ void put(void* p, V v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<V*>(p));
  else *reinterpret_cast<V*>(p) = v;
}
typedef uint32_t nt_u32x2 __attribute__((ext_vector_type(2)));

template <typename T, bool SPLIT, bool NT> __device__ __forceinline__ Raw8<T> ask8(const T* row, const Cols& at) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 4) {
    r.v[0] = __builtin_bit_cast(uint4, ask<nt_u32x4, NT>(row + at.a));
    r.v[1] = __builtin_bit_cast(uint4, ask<nt_u32x4, NT>(row + at.b));
  } else if constexpr (SPLIT) {
    const nt_u32x2 a = ask<nt_u32x2, NT>(row + at.a), b = ask<nt_u32x2, NT>(row + at.b);
    r.v[0] = make_uint4(a[0], a[1], b[0], b[1]);
  } else {
    r.v[0] = __builtin_bit_cast(uint4, ask<nt_u32x4, NT>(row + at.a));
  }
  return r;
}
template <typename T, bool SPLIT, bool NT> __device__ __forceinline__ void put8(T* row, const Cols& at, const f8& v) {
  Raw8<T> r;
  store8(reinterpret_cast<T*>(&r.v[0]), v);
  if constexpr (sizeof(T) == 4) {
    if (at.in_a) put<nt_u32x4, NT>(row + at.a, __builtin_bit_cast(nt_u32x4, r.v[0]));
    if (at.in_b) put<nt_u32x4, NT>(row + at.b, __builtin_bit_cast(nt_u32x4, r.v[1]));
  } else if constexpr (SPLIT) {
    if (at.in_a) put<nt_u32x2, NT>(row + at.a, nt_u32x2{r.v[0].x, r.v[0].y});
    if (at.in_b) put<nt_u32x2, NT>(row + at.b, nt_u32x2{r.v[0].z, r.v[0].w});
  } else {
    if (at.in_a) put<nt_u32x4, NT>(row + at.a, __builtin_bit_cast(nt_u32x4, r.v[0]));
  }
}
template <bool SPLIT, int P> __device__ __forceinline__ void weights(f8 (&w)[P], const float* wp, const Cols (&at)[P]) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    w[p] = raw_f8(ask8<float, SPLIT, false>(wp, at[p]));
#pragma unroll
    for (int j = 0; j < 8; ++j) w[p].v[j] += 1.f;
  }
}
// The parts of a sum over a piece that are in the row.
__device__ __forceinline__ float in_row(const Cols& at, float a, float b) {
  return (at.in_a ? a : 0.f) + (at.in_b ? b : 0.f);
}

template <typename T, typename R, bool MX8, int LPR, int P, int RB, bool NT, int MAXT>
__global__ void __launch_bounds__(MAXT) add_norm_fwd_kernel(AddNormArgs a) {
#pragma clang fp contract(off)
  constexpr bool SPLIT = sizeof(T) == 4 || sizeof(R) == 4;
  __shared__ float red[2][LPR == 64 ? 16 : 1][RB];
  const int waves = a.waves;                         // of a row; 1: rows of LPR lanes
  const int per = waves > 1 ? 1 : blockDim.x / LPR;  // rows side by side in a workgroup
  const int i = waves > 1 ? threadIdx.x : threadIdx.x % LPR;
  Cols at[P];
  cols<SPLIT, P>(at, i, waves > 1 ? blockDim.x : LPR, a.n);
  f8 w[P];
  weights<SPLIT, P>(w, a.w, at);
  const float inv = 1.f / (float)a.n;
  const int64_t step = (int64_t)gridDim.x * per * RB;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * per * RB; r0 < a.rows; r0 += step, turn ^= 1) {
    const int64_t r1 = r0 + (waves > 1 ? 0 : threadIdx.x / LPR);
    Raw8<T> x[RB][P];
    Raw8<R> s[RB][P];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int64_t r = r1 + b * per, rr = r < a.rows ? r : a.rows - 1;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        x[b][p] = ask8<T, SPLIT, NT>((const T*)a.x + rr * a.ldx, at[p]);
        if (a.res) s[b][p] = ask8<R, SPLIT, NT>((const R*)a.res + rr * a.ldr, at[p]);
      }
    }
    f8 v[RB][P];
    float ss[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      ss[b] = 0.f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        v[b][p] = raw_f8(x[b][p]);
        if (a.res) {
          const f8 u = raw_f8(s[b][p]);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[b][p].v[j] += u.v[j];
        }
        float qa = 0.f, qb = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          qa = fmaf(v[b][p].v[j], v[b][p].v[j], qa);
          qb = fmaf(v[b][p].v[j + 4], v[b][p].v[j + 4], qb);
        }
        ss[b] += in_row(at[p], qa, qb);
      }
    }
    row_sums<LPR, RB>(ss, red[turn], waves);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int64_t r = r1 + b * per;
      const float rho = rsqrtf(fmaf(ss[b], inv, a.eps));
      if (r < a.rows) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          if (a.h) put8<R, SPLIT, NT>((R*)a.h + r * a.ldh, at[p], v[b][p]);
          f8 y;
#pragma unroll
          for (int j = 0; j < 8; ++j) y.v[j] = v[b][p].v[j] * rho * w[p].v[j];
          // 8 bits: groups of 32 columns are 4 adjacent lanes, or 8 of each run.  They go
          // out in plain stores of 8 or 4 bytes a lane, which is near enough to the floor
          // (65536 x 2560 in bf16: 187 us for 176 us of bytes, fp32 32768 x 2560 167 for 163).
          if constexpr (MX8) {
            uint8_t* q = (uint8_t*)a.y + r * a.ldy;
            uint8_t* scale = a.scale + r * a.lds;
            float ma = amax4(y.v), mb = amax4(y.v + 4);
            if (!SPLIT) ma = mb = fmaxf(ma, mb);
            ma = fmaxf(ma, dpp_f<0xB1>(ma));
            ma = fmaxf(ma, dpp_f<0x4E>(ma));
            if (SPLIT) {
              ma = fmaxf(ma, dpp_f<0x141>(ma));
              mb = fmaxf(mb, dpp_f<0xB1>(mb));
              mb = fmaxf(mb, dpp_f<0x4E>(mb));
              mb = fmaxf(mb, dpp_f<0x141>(mb));
            }
            const int ea = mx8_exponent(ma), eb = SPLIT ? mx8_exponent(mb) : ea;
            const uint32_t wa = mx8_word(y.v, ea), wb = mx8_word(y.v + 4, eb);
            if constexpr (SPLIT) {
              if (at[p].in_a) {
                *(uint32_t*)(q + at[p].a) = wa;
                if (i % 8 == 0) scale[at[p].a / 32] = (uint8_t)(ea + 127);
              }
              if (at[p].in_b) {
                *(uint32_t*)(q + at[p].b) = wb;
                if (i % 8 == 0) scale[at[p].b / 32] = (uint8_t)(eb + 127);
              }
            } else if (at[p].in_a) {
              *(uint2*)(q + at[p].a) = make_uint2(wa, wb);
              if (i % 4 == 0) scale[at[p].a / 32] = (uint8_t)(ea + 127);
            }
          } else {
            put8<T, SPLIT, NT>((T*)a.y + r * a.ldy, at[p], y);
          }
        }
      }
    }
  }
}

// With n = h rho and dn = dy (1 + w):
//   d = dh + rho (dn - n mean(dn n)),  dw = sum over rows of dy n.
// A workgroup walks rows and keeps its dw in registers; the workgroups' partial
// sums are added in a fixed order.
template <typename T, typename R, int LPR, int P, int RB, bool NT, int MAXT, bool PF>
__global__ void __launch_bounds__(MAXT) add_norm_bwd_kernel(AddNormBwdArgs a) {
#pragma clang fp contract(off)
  constexpr bool SPLIT = sizeof(T) == 4 || sizeof(R) == 4;
  __shared__ float red[2][LPR == 64 ? 16 : 1][2 * RB];
  __shared__ float dws[MAXT == 256 ? 256 : 1][8 * P + 1];
  const int waves = a.waves;
  const int per = waves > 1 ? 1 : blockDim.x / LPR;
  const int i = waves > 1 ? threadIdx.x : threadIdx.x % LPR;
  Cols at[P];
  cols<SPLIT, P>(at, i, waves > 1 ? blockDim.x : LPR, a.n);
  f8 w[P], dw[P];
  if (P == 1) weights<SPLIT, P>(w, a.w, at);  // twice as many columns leave no registers: read where needed
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[p].v[j] = 0.f;
  const float inv = 1.f / (float)a.n;
  const int64_t step = (int64_t)gridDim.x * per * RB;
  int turn = 0;
  const int64_t first = (int64_t)blockIdx.x * per * RB + (waves > 1 ? 0 : threadIdx.x / LPR);
  struct Batch {
    Raw8<R> h[RB][P], up[RB][P];
    Raw8<T> dy[RB][P];
  } next;
  const auto ask = [&](Batch& to, int64_t r1) {
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int64_t r = r1 + b * per, rr = r < a.rows ? r : a.rows - 1;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        to.h[b][p] = ask8<R, SPLIT, NT>((const R*)a.h + rr * a.ldh, at[p]);
        to.dy[b][p] = ask8<T, SPLIT, NT>((const T*)a.dy + rr * a.lddy, at[p]);
        if (a.dh) to.up[b][p] = ask8<R, SPLIT, NT>((const R*)a.dh + rr * a.lddh, at[p]);
      }
    }
  };
  if (PF) ask(next, first);
  for (int64_t r0 = (int64_t)blockIdx.x * per * RB; r0 < a.rows; r0 += step, turn ^= 1) {
    const int64_t r1 = r0 + first - (int64_t)blockIdx.x * per * RB;
    Batch now;
    if (PF) {
      now = next;
      if (r0 + step < a.rows) ask(next, r1 + step);
    } else {
      ask(now, r1);
    }
    const auto& h = now.h;
    const auto& dy = now.dy;
    const auto& up = now.up;
    float sums[2 * RB];                // h^2 and dn h
    if (P > 1) weights<SPLIT, P>(w, a.w, at);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      sums[2 * b] = sums[2 * b + 1] = 0.f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const f8 hv = raw_f8(h[b][p]), dv = raw_f8(dy[b][p]);
        float qa = 0.f, qb = 0.f, ga = 0.f, gb = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          qa = fmaf(hv.v[j], hv.v[j], qa);
          ga = fmaf(dv.v[j] * w[p].v[j], hv.v[j], ga);
          qb = fmaf(hv.v[j + 4], hv.v[j + 4], qb);
          gb = fmaf(dv.v[j + 4] * w[p].v[j + 4], hv.v[j + 4], gb);
        }
        sums[2 * b] += in_row(at[p], qa, qb);
        sums[2 * b + 1] += in_row(at[p], ga, gb);
      }
    }
    row_sums<LPR, 2 * RB>(sums, red[turn], waves);
    if (P > 1) weights<SPLIT, P>(w, a.w, at);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int64_t r = r1 + b * per;
      const float rho = rsqrtf(fmaf(sums[2 * b], inv, a.eps));
      const float m = sums[2 * b + 1] * rho * inv;      // mean(dn n)
      if (r < a.rows) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const f8 hv = raw_f8(h[b][p]), dv = raw_f8(dy[b][p]);
          f8 d;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float n = hv.v[j] * rho;
            d.v[j] = rho * fmaf(-n, m, dv.v[j] * w[p].v[j]);
            dw[p].v[j] = fmaf(dv.v[j], n, dw[p].v[j]);
          }
          if (a.dh) {
            const f8 u = raw_f8(up[b][p]);
#pragma unroll
            for (int j = 0; j < 8; ++j) d.v[j] += u.v[j];
          }
          if (a.dx) put8<T, SPLIT, NT>((T*)a.dx + r * a.lddx, at[p], d);
          if (a.dres) put8<R, SPLIT, NT>((R*)a.dres + r * a.lddr, at[p], d);
        }
      }
    }
  }
  if (!a.partials) return;
  if constexpr (MAXT == 256) {         // rows side by side: their sums, in order
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int j = 0; j < 8; ++j) dws[threadIdx.x][8 * p + j] = dw[p].v[j];
    __syncthreads();
    if (threadIdx.x >= LPR) return;
    for (int u = 1; u < per; ++u)
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[p].v[j] += dws[u * LPR + i][8 * p + j];
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
    put8<float, SPLIT, false>(a.partials + (int64_t)blockIdx.x * a.n, at[p], dw[p]);
}

static int norm_waves(int n) { return n <= 512 ? 1 : n <= 8192 ? (n + 511) / 512 : 16; }
static int norm_lanes(int n) { return n <= 64 ? 8 : n <= 256 ? 32 : 64; }

// Workgroups of the backward: six to sixteen waves a CU (1024 workgroups of two
// waves at 1024 columns, 512 of three at 1032, 512 of eight at 4096, 256 of
// sixteen at 8192).  More only add partial sums of dw, fewer leave loads unasked.
// Where rows are taken two at a time and there are fewer than two for each
// workgroup, some workgroups get none and leave a partial sum of zeros.
// Measured, us by workgroups
// 256 / 512 / 1024: 16384 x 1000 - / 28 / 25, 16384 x 2560 - / 54.6 / 65,
// 3001 x 8192 34 / 38 / 43 (bf16).
int64_t add_norm_blocks(int64_t rows, int32_t n) {
  const int64_t per = n <= 512 ? 256 / norm_lanes(n) : 1, b = (rows + per - 1) / per;
  const int64_t most = n <= 1024 ? 1024 : n <= 4096 ? 512 : 256;
  return b < most ? b : most;
}

// Narrow rows: one at a time with the cache's help up to 1.5 times its 256 MB,
// beyond that as wide ones, from 65 columns on (narrower ones always one at a
// time).  262144 rows, us: bf16 x 128 (268 MB) 43.2, two at a time and
// non-temporal 44.3; bf16 x 256 93.2 and 86.1, fp32 x 512 382 and 362, its
// backward 439 and 378.
template <typename T, typename R> static bool beyond_cache(int64_t values) {
  return values * (int64_t)(sizeof(T) + sizeof(R)) * 2 >= (int64_t)3 << 27;
}

template <typename T, typename R, bool MX8, int LPR, int P, int RB, bool NT, int MAXT>
static hipError_t fwd_go(AddNormArgs a, hipStream_t st) {
  a.waves = norm_waves(a.n);
  const int threads = a.waves > 1 ? 64 * a.waves : 256, per = a.waves > 1 ? 1 : 256 / LPR;
  // one batch a workgroup; a launch holds fewer than 2^32 threads
  const int64_t b = (a.rows + per * RB - 1) / (per * RB), most = 1 << 21;
  hipLaunchKernelGGL((add_norm_fwd_kernel<T, R, MX8, LPR, P, RB, NT, MAXT>), dim3((unsigned)(b < most ? b : most)),
                     dim3(threads), 0, st, a);
  return hipGetLastError();
}

// Few rows: one at a time, for latency (16 rows of 2560: 2.9 us, two at a time
// 3.3).  Many: two at a time and non-temporal, since nothing of them is still
// cached when it is read again (65536 x 2560, bf16: one 220, two 210, four
// 216 us, two without the hint 259; a fixed grid that walks rows 224 to 247).
// Rows of more than eight waves one at a time (8192 x 8192: 88 us).
template <typename T, typename R, bool MX8>
static hipError_t fwd_n(const AddNormArgs& a, hipStream_t st) {
  const bool far = beyond_cache<T, R>(a.rows * a.n);
  if (a.n <= 64) return fwd_go<T, R, MX8, 8, 1, 1, false, 256>(a, st);
  if (a.n <= 256)
    return far ? fwd_go<T, R, MX8, 32, 1, 2, true, 256>(a, st)
               : fwd_go<T, R, MX8, 32, 1, 1, false, 256>(a, st);
  if (a.n <= 512)
    return far ? fwd_go<T, R, MX8, 64, 1, 2, true, 256>(a, st)
               : fwd_go<T, R, MX8, 64, 1, 1, false, 256>(a, st);
  if (a.n > 8192) return fwd_go<T, R, MX8, 64, 2, 1, true, 1024>(a, st);
  if (a.rows <= 2048) return fwd_go<T, R, MX8, 64, 1, 1, false, 1024>(a, st);
  if (a.n > 4096) return fwd_go<T, R, MX8, 64, 1, 1, true, 1024>(a, st);
  return fwd_go<T, R, MX8, 64, 1, 2, true, 512>(a, st);
}

template <typename T, typename R, int LPR, int P, int RB, bool NT, int MAXT, bool PF>
static hipError_t bwd_go(AddNormBwdArgs a, hipStream_t st) {
  a.waves = norm_waves(a.n);
  hipLaunchKernelGGL((add_norm_bwd_kernel<T, R, LPR, P, RB, NT, MAXT, PF>), dim3((unsigned)add_norm_blocks(a.rows, a.n)),
                     dim3(a.waves > 1 ? 64 * a.waves : 256), 0, st, a);
  return hipGetLastError();
}

// One workgroup of wide rows fills a CU, so that it has to ask for its next row
// itself (3001 x 8192: 34 us, 39 without); of narrower ones there are several,
// and two rows at a time are better (16384 x 2560: 54.6 us; one and the next
// 58.5, four 109).
template <typename T, typename R>
static hipError_t bwd_n(const AddNormBwdArgs& a, hipStream_t st) {
  const bool far = beyond_cache<T, R>(a.rows * a.n);
  if (a.n <= 64) return bwd_go<T, R, 8, 1, 1, false, 256, false>(a, st);
  if (a.n <= 256)
    return far ? bwd_go<T, R, 32, 1, 2, true, 256, false>(a, st)
               : bwd_go<T, R, 32, 1, 1, false, 256, false>(a, st);
  if (a.n <= 512)
    return far ? bwd_go<T, R, 64, 1, 2, true, 256, false>(a, st)
               : bwd_go<T, R, 64, 1, 1, false, 256, false>(a, st);
  if (a.n > 8192) return bwd_go<T, R, 64, 2, 1, true, 1024, false>(a, st);
  if (a.n > 4096) return bwd_go<T, R, 64, 1, 1, true, 1024, true>(a, st);
  return bwd_go<T, R, 64, 1, 2, true, 512, false>(a, st);
}

template <bool MX8> static hipError_t fwd_t(const AddNormArgs& a, hipStream_t st) {
  if (a.dtype == GDN_FP32) return fwd_n<float, float, MX8>(a, st);
  if (a.dtype == GDN_BF16)
    return a.res_dtype == GDN_FP32 ? fwd_n<bf16, float, MX8>(a, st) : fwd_n<bf16, bf16, MX8>(a, st);
  return a.res_dtype == GDN_FP32 ? fwd_n<fp16, float, MX8>(a, st) : fwd_n<fp16, fp16, MX8>(a, st);
}

hipError_t launch_add_norm_fwd(const AddNormArgs& a, hipStream_t st) {
  return a.scale ? fwd_t<true>(a, st) : fwd_t<false>(a, st);
}

hipError_t launch_add_norm_bwd(const AddNormBwdArgs& a, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (a.rows > 0) {
    if (a.dtype == GDN_FP32) e = bwd_n<float, float>(a, st);
    else if (a.dtype == GDN_BF16)
      e = a.res_dtype == GDN_FP32 ? bwd_n<bf16, float>(a, st) : bwd_n<bf16, bf16>(a, st);
    else
      e = a.res_dtype == GDN_FP32 ? bwd_n<fp16, float>(a, st) : bwd_n<fp16, fp16>(a, st);
  }
  if (e != hipSuccess || !a.dw) return e;
  return launch_reduce_partials(a.partials, add_norm_blocks(a.rows, a.n), a.n, a.dw, st);
}

}  // namespace gdn
