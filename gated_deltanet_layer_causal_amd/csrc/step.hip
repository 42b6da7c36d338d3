// The recurrent form of the layer core over cached states: the gated delta
// rule token by token (gdn_recurrent_fwd), and the whole core for the next
// tokens of every sequence (gdn_step_fwd).
//
// One workgroup owns one (sequence, value head).  The head's state S (D x D,
// fp32) stays in registers from its load to its store, so a call reads and
// writes each state once however many tokens a sequence has:
//   s = S_{t-1} k,  r = S_{t-1} q   (both from the old state, reduced together)
//   delta = beta (v - e^g s)
//   o = e^g r + delta (k . q),  S_t = e^g S_{t-1} + delta k^T
// which is the rule with o_t = S_t q_t expanded; q carries the scale.
//
// Tokens go through in blocks of STEP_TB: all threads form q, k, v (conv,
// SiLU, L2), e^g and beta of the block in LDS, then each thread walks the
// block's tokens for its part of the state, then all threads norm the block's
// outputs.
#include "chunk_common.h"
#include "launch.h"

namespace gdn {

constexpr int STEP_TB = 8;   // tokens per block

// Tokens of sequence n, clamped so that no table can lead outside [0, T].
__device__ __forceinline__ void token_range(const int32_t* cu, int n, int64_t T, int64_t& t0,
                                            int64_t& t1) {
  const int64_t a = cu[n], b = cu[n + 1];
  t0 = a < 0 ? 0 : a > T ? T : a;
  t1 = b < t0 ? t0 : b > T ? T : b;
}

__device__ __forceinline__ float softplus_full(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

// Sum over aligned groups of N lanes (2 for D = 32, 8 for D = 128).
template <int N> __device__ __forceinline__ float lanes_sum(float x) {
  if constexpr (N == 2) return x + dpp_f<0xB1>(x);
  else return lane_group_sum<N>(x);
}

// Thread layout of the state: LPR lanes share a row of D columns; a lane
// holds the columns 4 l + 4 LPR c + (0..3), c = 0..3, of R rows.
template <int D> struct StepGeo {
  static constexpr int LPR = D / 16;
  static constexpr int R = D == 128 ? 4 : 1;
  static constexpr int RPW = 64 / LPR;              // rows per wave and row slot
  static constexpr int WAVES = D / (RPW * R);
  static constexpr int THREADS = 64 * WAVES;
};

template <typename T, int D, bool STEP>
__global__ void __launch_bounds__(StepGeo<D>::THREADS) step_kernel(StepArgs p, int hk, int hv,
                                                                   int64_t T_tok) {
  typedef StepGeo<D> G;
  constexpr int NT = G::THREADS, G8 = D / 8;
  __shared__ float sq[STEP_TB][D], sk[STEP_TB][D], sv[STEP_TB][D];
  __shared__ float seg[STEP_TB], sbeta[STEP_TB];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = blockIdx.x / hv, h = blockIdx.x % hv, kh = h / (hv / hk);
  const int C = 2 * hk * D + hv * D;
  int64_t t0, t1;
  token_range(p.cu, n, T_tok, t0, t1);
  const int s_in = p.slot_in ? p.slot_in[n] : -1;
  const int s_out = p.slot_out ? p.slot_out[n] : -1;
  T* out = (T*)p.out;
  if (s_in >= p.cache.n_slots || s_out >= p.cache.n_slots) {   // a bad slot: NaN rows, no state
    for (int64_t i = tid; i < (t1 - t0) * D; i += NT)
      out[(t0 + i / D) * hv * D + (int64_t)h * D + i % D] = from_f<T>(__builtin_nanf(""));
    return;
  }
  if (t0 == t1 && (s_out < 0 || s_out == s_in)) return;

  const int row0 = wave * (G::RPW * G::R) + lane / G::LPR;
  const int col0 = 4 * (lane % G::LPR);
  float S[G::R][16];
  if (s_in >= 0) {
    const float* src = p.cache.S + (int64_t)s_in * p.cache.S_stride + (int64_t)h * D * D;
#pragma unroll
    for (int j = 0; j < G::R; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 v = *reinterpret_cast<const float4*>(src + (row0 + j * G::RPW) * D + col0 + 4 * G::LPR * c);
        S[j][4 * c] = v.x; S[j][4 * c + 1] = v.y; S[j][4 * c + 2] = v.z; S[j][4 * c + 3] = v.w;
      }
  } else {
#pragma unroll
    for (int j = 0; j < G::R; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) S[j][i] = 0.f;
  }
  auto put = [&](int slot) {
    float* dst = p.cache.S + (int64_t)slot * p.cache.S_stride + (int64_t)h * D * D;
#pragma unroll
    for (int j = 0; j < G::R; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<float4*>(dst + (row0 + j * G::RPW) * D + col0 + 4 * G::LPR * c) =
            make_float4(S[j][4 * c], S[j][4 * c + 1], S[j][4 * c + 2], S[j][4 * c + 3]);
  };

  for (int64_t tb = t0; tb < t1; tb += STEP_TB) {
    const int nt = t1 - tb < STEP_TB ? (int)(t1 - tb) : STEP_TB;
    // q, k, v of the block: job = (token, 8 channels of q, k or v)
    for (int job = tid; job < nt * 3 * G8; job += NT) {
      const int i = job / (3 * G8), part = job % (3 * G8) / G8, e = job % G8 * 8;
      const int64_t t = tb + i;
      f8 y;
      if constexpr (STEP) {
        const int ch = (part == 0 ? kh : part == 1 ? hk + kh : 2 * hk + h) * D + e;
        float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t tr = t - 3 + j;
          f8 xr;
          if (tr >= t0) {
            xr = load8((const T*)p.x + tr * p.ldx + ch);
          } else if (s_in >= 0) {
            xr = load8((const T*)p.cache.conv + (int64_t)s_in * p.cache.conv_stride +
                       (tr - t0 + 3) * C + ch);
          } else {
#pragma unroll
            for (int m = 0; m < 8; ++m) xr.v[m] = 0.f;
          }
#pragma unroll
          for (int m = 0; m < 8; ++m) u[m] += p.w_conv[(int64_t)(ch + m) * 4 + j] * xr.v[m];
        }
        float sq2 = 0.f;
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          y.v[m] = u[m] * sigmoidf_(u[m]);
          sq2 += y.v[m] * y.v[m];
        }
        sq2 = lane_group_sum<G8>(sq2);
        const float r = part == 2 ? 1.f : rsqrtf(sq2 + p.l2_eps) * (part == 0 ? p.scale : 1.f);
#pragma unroll
        for (int m = 0; m < 8; ++m) y.v[m] *= r;
      } else {
        y = part == 0   ? load8((const T*)p.q + t * p.ldq + kh * D + e)
            : part == 1 ? load8((const T*)p.k + t * p.ldk + kh * D + e)
                        : load8((const T*)p.v + t * p.ldv + h * D + e);
        if (part == 0) {
#pragma unroll
          for (int m = 0; m < 8; ++m) y.v[m] *= p.scale;
        }
      }
      store8(part == 0 ? &sq[i][e] : part == 1 ? &sk[i][e] : &sv[i][e], y);
    }
    if (tid < nt) {
      const int64_t t = tb + tid;
      if constexpr (STEP) {
        const float xa = to_f(((const T*)p.a)[t * p.lda + h]) + p.dt_bias[h];
        seg[tid] = expf(-expf(p.A_log[h]) * softplus_full(xa));
        sbeta[tid] = sigmoidf_(to_f(((const T*)p.b)[t * p.ldb + h]));
      } else {
        seg[tid] = expf(p.g[t * hv + h]);
        sbeta[tid] = p.beta[t * hv + h];
      }
    }
    __syncthreads();
    for (int i = 0; i < nt; ++i) {
      float k[16], q[16];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 a = *reinterpret_cast<const float4*>(&sk[i][col0 + 4 * G::LPR * c]);
        const float4 b = *reinterpret_cast<const float4*>(&sq[i][col0 + 4 * G::LPR * c]);
        k[4 * c] = a.x; k[4 * c + 1] = a.y; k[4 * c + 2] = a.z; k[4 * c + 3] = a.w;
        q[4 * c] = b.x; q[4 * c + 1] = b.y; q[4 * c + 2] = b.z; q[4 * c + 3] = b.w;
      }
      float kq = 0.f, s[G::R], r[G::R];
#pragma unroll
      for (int m = 0; m < 16; ++m) kq += k[m] * q[m];
#pragma unroll
      for (int j = 0; j < G::R; ++j) {
        s[j] = r[j] = 0.f;
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          s[j] += S[j][m] * k[m];
          r[j] += S[j][m] * q[m];
        }
      }
      kq = lanes_sum<G::LPR>(kq);
      const float eg = seg[i], beta = sbeta[i];
#pragma unroll
      for (int j = 0; j < G::R; ++j) {
        const int row = row0 + j * G::RPW;
        const float sj = lanes_sum<G::LPR>(s[j]), rj = lanes_sum<G::LPR>(r[j]);
        const float delta = beta * (sv[i][row] - eg * sj);
#pragma unroll
        for (int m = 0; m < 16; ++m) S[j][m] = eg * S[j][m] + delta * k[m];
        // only this row's lanes, of one wave, read sv[i][row]: o takes its place
        if (lane % G::LPR == 0) sv[i][row] = eg * rj + delta * kq;
      }
      if (p.slot_tok) {
        const int st = p.slot_tok[tb + i];
        if (st >= 0 && st < p.cache.n_slots) put(st);
      }
    }
    __syncthreads();
    for (int job = tid; job < nt * G8; job += NT) {
      const int i = job / G8, e = job % G8 * 8;
      const int64_t t = tb + i;
      f8 o = load8(&sv[i][e]);
      if constexpr (STEP) {
        float ss = 0.f;
#pragma unroll
        for (int m = 0; m < 8; ++m) ss += o.v[m] * o.v[m];
        ss = lane_group_sum<G8>(ss);
        const float rho = rsqrtf(ss * (1.f / D) + p.norm_eps);
        const f8 z = load8((const T*)p.z + t * p.ldz + h * D + e);
        const f8 w = load8(p.w_norm + e);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const float sg = sigmoidf_(z.v[m]);
          o.v[m] *= rho * (1.f + w.v[m]) * (p.act == 0 ? z.v[m] * sg : sg);
        }
      }
      store8(out + t * hv * D + h * D + e, o);
    }
    __syncthreads();
  }
  if (s_out >= 0) put(s_out);
}

// The conv rows of the states: after token t the last three input rows are
// x[t-2], x[t-1], x[t], reaching back into the rows of slot_in.  A second
// launch, since several heads' workgroups of the step read those rows.  A
// thread owns 8 channels of one sequence and reads the rows it needs before
// it writes any, so that slots may be updated in place.
template <typename T>
__global__ void __launch_bounds__(256) step_rows_kernel(StepArgs p, int n_grp, int64_t T_tok) {
  const int n = blockIdx.y, grp = blockIdx.x * 256 + threadIdx.x;
  if (grp >= n_grp) return;
  int64_t t0, t1;
  token_range(p.cu, n, T_tok, t0, t1);
  const int s_in = p.slot_in ? p.slot_in[n] : -1;
  const int s_out = p.slot_out ? p.slot_out[n] : -1;
  if (s_in >= p.cache.n_slots || s_out >= p.cache.n_slots) return;
  const int64_t C = (int64_t)n_grp * 8;
  const T* x = (const T*)p.x + grp * 8;
  T* rows = (T*)p.cache.conv + grp * 8;
  Raw8<T> w[3];
#pragma unroll
  for (int j = 0; j < 3; ++j)
    w[j] = s_in >= 0 ? ld_raw8(rows + (int64_t)s_in * p.cache.conv_stride + j * C) : zero_raw8<T>();
  auto put = [&](int slot) {
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
      for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
        reinterpret_cast<uint4*>(rows + (int64_t)slot * p.cache.conv_stride + j * C)[i] = w[j].v[i];
  };
  // without tables for single tokens only the last three rows matter
  const int64_t tb = p.slot_tok || t1 - t0 < 3 ? t0 : t1 - 3;
  for (int64_t t = tb; t < t1; ++t) {
    w[0] = w[1];
    w[1] = w[2];
    w[2] = ld_raw8(x + t * p.ldx);
    if (p.slot_tok) {
      const int st = p.slot_tok[t];
      if (st >= 0 && st < p.cache.n_slots) put(st);
    }
  }
  if (s_out >= 0 && (t1 > t0 || s_out != s_in)) put(s_out);
}

template <typename T, bool STEP>
static void launch_step_d(const gdn_shape& s, const StepArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)s.n_seq * (unsigned)s.hv);
  if (s.dk == 128)
    hipLaunchKernelGGL((step_kernel<T, 128, STEP>), grid, dim3(StepGeo<128>::THREADS), 0, st, a,
                       s.hk, s.hv, s.total_tokens);
  else
    hipLaunchKernelGGL((step_kernel<T, 32, STEP>), grid, dim3(StepGeo<32>::THREADS), 0, st, a, s.hk,
                       s.hv, s.total_tokens);
}

hipError_t launch_recurrent(const gdn_shape& s, const StepArgs& a, hipStream_t st) {
  if (s.dtype == GDN_BF16) launch_step_d<bf16, false>(s, a, st);
  else if (s.dtype == GDN_FP16) launch_step_d<fp16, false>(s, a, st);
  else launch_step_d<float, false>(s, a, st);
  return hipGetLastError();
}

template <typename T>
static hipError_t launch_step_t(const gdn_shape& s, const StepArgs& a, hipStream_t st) {
  launch_step_d<T, true>(s, a, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!a.slot_out && !a.slot_tok)) return e;
  const int n_grp = (2 * s.hk * s.dk + s.hv * s.dv) / 8;
  hipLaunchKernelGGL((step_rows_kernel<T>), dim3((n_grp + 255) / 256, s.n_seq), dim3(256), 0, st, a,
                     n_grp, s.total_tokens);
  return hipGetLastError();
}

hipError_t launch_step(const gdn_shape& s, const StepArgs& a, hipStream_t st) {
  if (s.dtype == GDN_BF16) return launch_step_t<bf16>(s, a, st);
  if (s.dtype == GDN_FP16) return launch_step_t<fp16>(s, a, st);
  return launch_step_t<float>(s, a, st);
}

// Check of the slot tables, one workgroup: a table of each slot's writing
// sequence in LDS, for a range of slots at a time.
constexpr int CHECK_RANGE = 8192;
__global__ void __launch_bounds__(256) check_slots_kernel(const int32_t* __restrict__ cu, int n_seq,
                                                          int64_t T_tok, int n_slots,
                                                          const int32_t* __restrict__ slot_in,
                                                          const int32_t* __restrict__ slot_out,
                                                          const int32_t* __restrict__ slot_tok,
                                                          int32_t* __restrict__ out) {
  __shared__ int32_t writer[CHECK_RANGE];
  __shared__ int32_t acc;
  if (threadIdx.x == 0) acc = 0;
  int32_t bad = 0;
  for (int64_t lo = 0; lo < n_slots; lo += CHECK_RANGE) {
    __syncthreads();
    for (int i = threadIdx.x; i < CHECK_RANGE; i += 256) writer[i] = -1;
    __syncthreads();
    auto claim = [&](int slot, int n) {
      if (slot >= n_slots) bad |= 1;
      else if (slot >= lo && slot < lo + CHECK_RANGE && atomicCAS(&writer[slot - lo], -1, n) != -1) bad |= 2;
    };
    for (int n = threadIdx.x; n < n_seq; n += 256) {
      int64_t t0, t1;
      token_range(cu, n, T_tok, t0, t1);
      if (slot_out) claim(slot_out[n], n);
      if (slot_tok)
        for (int64_t t = t0; t < t1; ++t) claim(slot_tok[t], n);
    }
    __syncthreads();
    if (slot_in)
      for (int n = threadIdx.x; n < n_seq; n += 256) {
        const int slot = slot_in[n];
        if (slot >= n_slots) bad |= 1;
        else if (slot >= lo && slot < lo + CHECK_RANGE && writer[slot - lo] != -1 && writer[slot - lo] != n) bad |= 4;
      }
  }
  __syncthreads();
  if (bad) atomicOr(&acc, bad);
  __syncthreads();
  if (threadIdx.x == 0) out[0] = acc;
}

hipError_t launch_check_slots(const gdn_shape& s, int32_t n_slots, const int32_t* slot_in,
                              const int32_t* slot_out, const int32_t* slot_tok, const int32_t* cu,
                              int32_t* out, hipStream_t st) {
  hipLaunchKernelGGL(check_slots_kernel, dim3(1), dim3(256), 0, st, cu, s.n_seq, s.total_tokens,
                     n_slots, slot_in, slot_out, slot_tok, out);
  return hipGetLastError();
}

}  // namespace gdn
