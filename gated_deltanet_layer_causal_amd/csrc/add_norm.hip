// The residual's addition with the zero-centred RMSNorm that follows it:
//   h = x + res,  y = h * rho * (1 + w),  rho = (mean h^2 + eps)^(-1/2)
// and its backward.  HBM-bound: each row is read once, held in registers and
// written once.  The norm reads the sum before h is rounded to its storage
// type, so y carries one rounding.
#include "common.h"
#include "launch.h"

namespace gdn {

// A row is owned by TPR threads (WPR waves); thread i of them holds the 8
// columns at (p * TPR + i) * 8 of each piece p < P.
template <int WPR>
__device__ __forceinline__ float group_sum(float x, float* red) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m);
  if constexpr (WPR > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) x += red[wave / WPR * WPR + i];
  }
  return x;
}

// 8 values of a group of 32 columns (4 adjacent lanes) in e4m3 under the
// smallest power of two that keeps the group within 448 = 0.875 * 2^9.
// NaN stays NaN and leaves the scale to the others; infinities become NaN.
__device__ __forceinline__ uint2 to_mx8(const f8& v, int* scale) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v.v[i]));
  amax = fmaxf(amax, dpp_f<0xB1>(amax));
  amax = fmaxf(amax, dpp_f<0x4E>(amax));
  int e = __builtin_amdgcn_frexp_expf(amax) - 9 + (__builtin_amdgcn_frexp_mantf(amax) > 0.875f);
  if (amax == 0.f) e = -127;
  if (__builtin_isinf(amax)) e = 127;
  e = e < -127 ? -127 : e > 127 ? 127 : e;
  *scale = e + 127;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = ldexpf(v.v[i], -e);
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

template <typename T, typename R, bool MX8, int WPR, int P>
__global__ void __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) add_norm_fwd_kernel(AddNormArgs a) {
  constexpr int TPR = 64 * WPR, GROUPS = WPR == 1 ? 4 : 1;
  __shared__ float red[WPR == 1 ? 1 : WPR];
  const int i = threadIdx.x % TPR;
  const int64_t r = (int64_t)blockIdx.x * GROUPS + threadIdx.x / TPR;
  if (r >= a.rows) return;       // a whole row's threads: no barrier is missed
  const T* x = (const T*)a.x + r * a.ldx;
  const R* res = (const R*)a.res + r * a.ldr;
  f8 v[P];
  float ss = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = (p * TPR + i) * 8;
    if (c < a.n) {
      v[p] = load8(x + c);
      if (a.res) {
        const f8 s = load8(res + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[p].v[j] += s.v[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += v[p].v[j] * v[p].v[j];
    }
  }
  ss = group_sum<WPR>(ss, red);
  const float rho = rsqrtf(ss / (float)a.n + a.eps);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = (p * TPR + i) * 8;
    if (c < a.n) {
      if (a.h) store8((R*)a.h + r * a.ldh + c, v[p]);
      const f8 w = load8(a.w + c);
      f8 y;
#pragma unroll
      for (int j = 0; j < 8; ++j) y.v[j] = v[p].v[j] * rho * (1.f + w.v[j]);
      if constexpr (MX8) {
        int e;
        const uint2 q = to_mx8(y, &e);
        *(uint2*)((uint8_t*)a.y + r * a.ldy + c) = q;
        if (i % 4 == 0) a.scale[r * a.lds + c / 32] = (uint8_t)e;
      } else {
        store8((T*)a.y + r * a.ldy + c, y);
      }
    }
  }
}

// With n = h rho and dn = dy (1 + w):
//   d = dh + rho (dn - n mean(dn n)),  dw = sum over rows of dy n.
// A block walks rows and keeps its dw in registers; the blocks' partial sums
// are added in a fixed order.
template <typename T, typename R, int WPR, int P>
__global__ void __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) add_norm_bwd_kernel(AddNormBwdArgs a) {
  constexpr int TPR = 64 * WPR, GROUPS = WPR == 1 ? 4 : 1;
  __shared__ float red[2][WPR == 1 ? 1 : WPR];
  __shared__ float4 dws[GROUPS == 1 ? 1 : 3][GROUPS == 1 ? 1 : 2][TPR];
  const int i = threadIdx.x % TPR, g = threadIdx.x / TPR;
  f8 dw[P];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[p].v[j] = 0.f;
  for (int64_t r = (int64_t)blockIdx.x * GROUPS + g; r < a.rows; r += (int64_t)gridDim.x * GROUPS) {
    const R* h = (const R*)a.h + r * a.ldh;
    const T* dy = (const T*)a.dy + r * a.lddy;
    f8 hv[P], dv[P];
    float ss = 0.f, sd = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * TPR + i) * 8;
      if (c < a.n) {
        hv[p] = load8(h + c);
        dv[p] = load8(dy + c);
        const f8 w = load8(a.w + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss += hv[p].v[j] * hv[p].v[j];
          sd += dv[p].v[j] * (1.f + w.v[j]) * hv[p].v[j];
        }
      }
    }
    ss = group_sum<WPR>(ss, red[0]);
    sd = group_sum<WPR>(sd, red[1]);
    const float rho = rsqrtf(ss / (float)a.n + a.eps);
    const float m = sd * rho / (float)a.n;     // mean(dn n)
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * TPR + i) * 8;
      if (c < a.n) {
        const f8 w = load8(a.w + c);
        f8 d;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float n = hv[p].v[j] * rho;
          d.v[j] = rho * (dv[p].v[j] * (1.f + w.v[j]) - n * m);
          dw[p].v[j] += dv[p].v[j] * n;
        }
        if (a.dh) {
          const f8 u = load8((const R*)a.dh + r * a.lddh + c);
#pragma unroll
          for (int j = 0; j < 8; ++j) d.v[j] += u.v[j];
        }
        if (a.dx) store8((T*)a.dx + r * a.lddx + c, d);
        if (a.dres) store8((R*)a.dres + r * a.lddr + c, d);
      }
    }
    if constexpr (WPR > 1) __syncthreads();    // red is written again
  }
  if (!a.partials) return;
  if constexpr (GROUPS > 1) {                  // the four waves' sums, in wave order
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (g > 0) {
        dws[g - 1][0][i] = make_float4(dw[p].v[0], dw[p].v[1], dw[p].v[2], dw[p].v[3]);
        dws[g - 1][1][i] = make_float4(dw[p].v[4], dw[p].v[5], dw[p].v[6], dw[p].v[7]);
      }
      __syncthreads();
      if (g == 0) {
#pragma unroll
        for (int k = 0; k < GROUPS - 1; ++k) {
          const float4 lo = dws[k][0][i], hi = dws[k][1][i];
          dw[p].v[0] += lo.x; dw[p].v[1] += lo.y; dw[p].v[2] += lo.z; dw[p].v[3] += lo.w;
          dw[p].v[4] += hi.x; dw[p].v[5] += hi.y; dw[p].v[6] += hi.z; dw[p].v[7] += hi.w;
        }
      }
      __syncthreads();
    }
  }
  if (g == 0) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int c = (p * TPR + i) * 8;
      if (c < a.n) store8(a.partials + (int64_t)blockIdx.x * a.n + c, dw[p]);
    }
  }
}

int64_t add_norm_blocks(int64_t rows, int32_t n) {
  const int64_t b = n <= ADD_NORM_WAVE ? (rows + 3) / 4 : rows;
  return b < ADD_NORM_BLOCKS_MAX ? b : ADD_NORM_BLOCKS_MAX;
}

template <typename T, typename R, bool MX8, int WPR, int P>
static hipError_t fwd_go(const AddNormArgs& a, hipStream_t st) {
  // a launch holds fewer than 2^32 threads
  constexpr int64_t G = WPR == 1 ? 4 : 1, STEP = (int64_t)1 << 20;
  for (int64_t r0 = 0; r0 < a.rows; r0 += STEP) {
    AddNormArgs b = a;
    b.rows = a.rows - r0 < STEP ? a.rows - r0 : STEP;
    b.x = (const T*)a.x + r0 * a.ldx;
    if (a.res) b.res = (const R*)a.res + r0 * a.ldr;
    if (a.h) b.h = (R*)a.h + r0 * a.ldh;
    b.y = MX8 ? (void*)((uint8_t*)a.y + r0 * a.ldy) : (void*)((T*)a.y + r0 * a.ldy);
    if (MX8) b.scale = a.scale + r0 * a.lds;
    hipLaunchKernelGGL((add_norm_fwd_kernel<T, R, MX8, WPR, P>), dim3((unsigned)((b.rows + G - 1) / G)),
                       dim3(WPR == 1 ? 256 : 64 * WPR), 0, st, b);
  }
  return hipGetLastError();
}

template <typename T, typename R, bool MX8>
static hipError_t fwd_n(const AddNormArgs& a, hipStream_t st) {
  if (a.n <= 1024) return fwd_go<T, R, MX8, 1, 2>(a, st);
  if (a.n <= ADD_NORM_WAVE) return fwd_go<T, R, MX8, 1, 5>(a, st);
  if (a.n <= 8192) return fwd_go<T, R, MX8, 4, 4>(a, st);
  return fwd_go<T, R, MX8, 16, 2>(a, st);
}

template <typename T, typename R, int WPR, int P>
static hipError_t bwd_go(const AddNormBwdArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((add_norm_bwd_kernel<T, R, WPR, P>), dim3((unsigned)add_norm_blocks(a.rows, a.n)),
                     dim3(WPR == 1 ? 256 : 64 * WPR), 0, st, a);
  return hipGetLastError();
}

template <typename T, typename R>
static hipError_t bwd_n(const AddNormBwdArgs& a, hipStream_t st) {
  if (a.n <= 1024) return bwd_go<T, R, 1, 2>(a, st);
  if (a.n <= ADD_NORM_WAVE) return bwd_go<T, R, 1, 5>(a, st);
  if (a.n <= 8192) return bwd_go<T, R, 4, 4>(a, st);
  return bwd_go<T, R, 16, 2>(a, st);
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
