// The recurrent form of the layer core over cached states: the gated delta
// rule token by token (gdn_recurrent_fwd), and the whole core for the next
// tokens of every sequence (gdn_step_fwd).
//
// One workgroup owns one sequence and some value heads of one key head.  The
// step takes all of them, HW at a time, so that it alone reads and writes
// their conv rows (or one, and a second launch writes the rows of q and k).
// The rule takes one, or a quarter of one's rows: the rows of S share nothing
// but k and q.  A head's state S (D x D, fp32) stays in registers from its
// load to its store, so a call reads and writes each state once however many
// tokens a sequence has:
//   s = S_{t-1} k,  r = S_{t-1} q   (both from the old state, reduced together)
//   delta = beta (v - e^g s)
//   o = e^g r + delta (k . q),  S_t = e^g S_{t-1} + delta k^T
// which is the rule with o_t = S_t q_t expanded; q carries the scale.
//
// The state waves do only that.  The helper waves form q, k, v (conv, SiLU,
// L2), e^g and beta of a block of STEP_TB tokens in LDS while the state waves
// load the state or walk the block before, and norm and store the outputs of
// the block behind them: neither their loads nor their arithmetic sit between
// a state's load and its store.  One barrier per block joins the two; the
// blocks of q and k alternate between two buffers, those of v (and o, which
// takes its place) between two or, with more than one helper wave, three.
#include "chunk_stream.h"
#include "launch.h"

namespace gdn {

constexpr int STEP_TB = 8;             // tokens per block
constexpr unsigned STEP_THROUGH = 128; // workgroups from which states are written through: a
                                       // loss at 16, a gain at thousands, no difference at 148
                                       // (11.5 against 11.7 us, the spread of one side's runs)

// Tokens of sequence n, clamped so that no table can lead outside [0, T].
__device__ __forceinline__ void token_range(const int32_t* cu, int n, int T, int& t0, int& t1) {
  const int a = __builtin_amdgcn_readfirstlane(cu[n]), b = __builtin_amdgcn_readfirstlane(cu[n + 1]);
  t0 = a < 0 ? 0 : a > T ? T : a;
  t1 = b < t0 ? t0 : b > T ? T : b;
}
// Entry n of a slot table (uniform n); -1 without one.
__device__ __forceinline__ int slot_of(const int32_t* table, int n) {
  return table ? __builtin_amdgcn_readfirstlane(table[n]) : -1;
}

__device__ __forceinline__ float softplus_full(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

__device__ __forceinline__ float lane_of(float x, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), l));
}

// Between LDS reads of some lanes of a wave and writes of others to the same
// words: a wave's LDS operations take effect in order, so only the compiler has
// to keep them so (no instruction comes of it).
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Thread layout of the state: LPR lanes share a row of D columns; a lane
// holds the columns 4 l + 4 LPR c + (0..3), c = 0 .. NC - 1, of R rows, so
// that the lanes of a row touch whole 128-byte lines at a time (with two
// lanes a row at D = 32, 32 bytes of each line, the rule took 125 us instead
// of 32 us for 254 sequences x 48 heads with every state kept twice).  SPLIT
// workgroups share a head, VC value rows each; R < 4 / SPLIT spreads them over
// more waves.
template <int D, int HW, int SPLIT, int R_ = 4 / SPLIT> struct StepGeo {
  static constexpr int LPR = 8, NC = D / (4 * LPR);
  static constexpr int R = R_;
  static constexpr int RPW = 64 / LPR;              // rows per wave and row slot
  static constexpr int VC = D / SPLIT;
  static constexpr int WAVES = VC / (RPW * R);      // state waves of a head
  // helper lanes: 8 channels each of q, k and HW times v, then a gate each
  static constexpr int CONV_LANES = (2 * D + HW * VC) / 8, HELPERS = (CONV_LANES + HW * STEP_TB + 63) / 64;
  static constexpr int THREADS = 64 * (HW * WAVES + HELPERS);
};

template <int D, int HW, int SPLIT> struct StepLds {
  // One helper wave takes o out of v's buffer before it puts the block after
  // next there; of several, one could be a step ahead: a third buffer.
  static constexpr int NV = StepGeo<D, HW, SPLIT>::HELPERS > 1 ? 3 : 2;
  float q[2][STEP_TB][D], k[2][STEP_TB][D];
  float v[NV][HW][STEP_TB][D / SPLIT];                              // v, then o in its place
  float eg[2][HW][STEP_TB], beta[2][HW][STEP_TB];
  int tok[2][STEP_TB];                                              // slot_tok, -1: none
};

// What a workgroup works on: value heads h0 .. h1 - 1 of key head kh, HW at a
// time (a round), each round in nb blocks of STEP_TB tokens; item i = (round
// i / nb, block i % nb).  v0: the first value row of those that share a head.
struct StepSpan {
  int t0, t1, s_in, s_out, h0, h1, kh, nb, items, v0;
  bool all;   // all heads of kh are here
};

// A head's state: its load, its tokens, its store.
template <int D, int SPLIT, int R> struct StepState {
  typedef StepGeo<D, 1, SPLIT, R> G;
  floatx4 S[G::R][G::NC];
  uint32_t row0, col0, at;   // first row of the workgroup's, first column, and their byte in S

  __device__ __forceinline__ StepState(int wave, int lane, int v0)
      : row0(wave * (G::RPW * G::R) + lane / G::LPR), col0(4 * (lane % G::LPR)),
        at(4 * ((v0 + row0) * D + col0)) {}

  // Each state passes through once, in whole lines: non-temporal both ways (the
  // rule, 200 sequences x 48 heads, bf16: 251 us with plain accesses, 245 us
  // with the hint on one side, 220 us on both).  Stores that are written
  // through as well (sc1) are faster where the chip is full (212 us) and
  // slower from a few workgroups (the step, one sequence x 48 heads: 9.3 us
  // without, 11.8 us with); see STEP_THROUGH.
  __device__ __forceinline__ static __amdgpu_buffer_rsrc_t head(const StepArgs& p, int slot, int h) {
    return buffer_of(p.cache.S + (int64_t)slot * p.cache.S_stride + (int64_t)h * D * D, 4 * D * D);
  }
  __device__ __forceinline__ void load(const StepArgs& p, int slot, int h) {
    if (slot >= 0) {
      const auto rs = head(p, slot, h);
#pragma unroll
      for (int j = 0; j < G::R; ++j)
#pragma unroll
        for (int c = 0; c < G::NC; ++c)
          S[j][c] = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(
              rs, at + 16 * G::LPR * c, 4 * j * G::RPW * D, CACHE_NT));
    } else {
#pragma unroll
      for (int j = 0; j < G::R; ++j)
#pragma unroll
        for (int c = 0; c < G::NC; ++c) S[j][c] = zero4();
    }
  }
  template <int AUX>
  __device__ __forceinline__ void store_as(const __amdgpu_buffer_rsrc_t rs) const {
#pragma unroll
    for (int j = 0; j < G::R; ++j)
#pragma unroll
      for (int c = 0; c < G::NC; ++c)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[j][c]), rs, at + 16 * G::LPR * c,
                                               4 * j * G::RPW * D, AUX);
  }
  __device__ __forceinline__ void store(const StepArgs& p, int slot, int h) const {
    const auto rs = head(p, slot, h);
    if (p.through) store_as<CACHE_NT | CACHE_SC1>(rs);
    else store_as<CACHE_NT>(rs);
  }
  // k . q of a whole block, token lane / 8 in each lane, instead of each
  // token's in every group of lanes; summed in the same order.  The rule takes
  // it so, and the step of long pieces with eight waves a head: 512 tokens of 48 heads 145 us against 157 us, 7 sequences of up to
  // 97 tokens x 32 heads 38 us against 40 us.  In the step's short calls it
  // would only stand between a barrier and the first token (64 sequences 81.4
  // against 80.5 us, 384 sequences 428 against 426.5 us).
  __device__ __forceinline__ static float block_kq(const float (*sq)[D], const float (*sk)[D], int lane) {
    static_assert(G::LPR * STEP_TB == 64, "a token to each group of lanes");
    const int t = lane / G::LPR, at = 4 * (lane % G::LPR);
    float kq = 0.f;
#pragma unroll
    for (int c = 0; c < G::NC; ++c) {
      const floatx4 k = *reinterpret_cast<const floatx4*>(&sk[t][at + 4 * G::LPR * c]);
      const floatx4 q = *reinterpret_cast<const floatx4*>(&sq[t][at + 4 * G::LPR * c]);
#pragma unroll
      for (int m = 0; m < 4; ++m) kq = fmaf(k[m], q[m], kq);
    }
    return lane_group_sum<G::LPR>(kq);
  }
  // One token; its outputs take the place of v.  k and q pass through
  // registers 4 columns at a time.  k stays for the update where a lane has
  // few elements of the state (512 tokens of 48 heads: 145 us, read again
  // 155 us) and is read again beside 64, where it would not fit.  kq: k . q,
  // where the block's are formed.
  template <bool BLOCK_KQ>
  __device__ __forceinline__ void token(const float* sq, const float* sk, float* sv, float eg,
                                        float beta, float kq, int lane) {
    constexpr bool K_STAYS = G::R * G::NC <= 4;
    float s[G::R], r[G::R], v[G::R];
    floatx4 kk[G::NC];
#pragma unroll
    for (int j = 0; j < G::R; ++j) {
      s[j] = r[j] = 0.f;
      v[j] = sv[row0 + j * G::RPW];
    }
#pragma unroll
    for (int c = 0; c < G::NC; ++c) {
      const floatx4 k = *reinterpret_cast<const floatx4*>(sk + col0 + 4 * G::LPR * c);
      if (K_STAYS) kk[c] = k;
      const floatx4 q = *reinterpret_cast<const floatx4*>(sq + col0 + 4 * G::LPR * c);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (!BLOCK_KQ) kq = fmaf(k[m], q[m], kq);
#pragma unroll
        for (int j = 0; j < G::R; ++j) {
          s[j] = fmaf(S[j][c][m], k[m], s[j]);
          r[j] = fmaf(S[j][c][m], q[m], r[j]);
        }
      }
    }
    if (!BLOCK_KQ) kq = lane_group_sum<G::LPR>(kq);
#pragma unroll
    for (int j = 0; j < G::R; ++j) {
      s[j] = lane_group_sum<G::LPR>(s[j]);
      r[j] = lane_group_sum<G::LPR>(r[j]);
    }
#pragma unroll
    for (int j = 0; j < G::R; ++j) {
      s[j] = beta * (v[j] - eg * s[j]);        // delta
      r[j] = fmaf(s[j], kq, eg * r[j]);        // o
    }
    if (lane % G::LPR == 0) {                  // only a row's own lanes read its v
#pragma unroll
      for (int j = 0; j < G::R; ++j) sv[row0 + j * G::RPW] = r[j];
    }
#pragma unroll
    for (int c = 0; c < G::NC; ++c) {
      const floatx4 k = K_STAYS ? kk[c] : *reinterpret_cast<const floatx4*>(sk + col0 + 4 * G::LPR * c);
#pragma unroll
      for (int j = 0; j < G::R; ++j)
#pragma unroll
        for (int m = 0; m < 4; ++m) S[j][c][m] = fmaf(s[j], k[m], eg * S[j][c][m]);
    }
  }
};

template <int D, int HW, int SPLIT, bool BLOCK_KQ, int R>
__device__ __forceinline__ void step_state_wave(const StepArgs& p, const StepSpan& w,
                                                StepLds<D, HW, SPLIT>& lds, int wave, int lane) {
  constexpr int WAVES = StepGeo<D, HW, SPLIT, R>::WAVES;
  const int hw = wave / WAVES;                    // which of the round's heads
  StepState<D, SPLIT, R> st(wave % WAVES, lane, w.v0);
  int h = w.h0 + hw, blk = 0;
  if (h < w.h1) st.load(p, w.s_in, h);
  for (int i = 0; i < w.items; ++i) {
    const int buf = i & 1, vb = i % StepLds<D, HW, SPLIT>::NV;
    const int left = w.t1 - w.t0 - blk * STEP_TB;
    const int nt = h >= w.h1 ? 0 : left < STEP_TB ? left : STEP_TB;
    __syncthreads();   // q, k, v of item i are in LDS
    const float kq = !BLOCK_KQ ? 0.f : StepState<D, SPLIT, R>::block_kq(lds.q[buf], lds.k[buf], lane);
    for (int j = 0; j < nt; ++j) {
      st.template token<BLOCK_KQ>(lds.q[buf][j], lds.k[buf][j], lds.v[vb][hw][j], lds.eg[buf][hw][j],
                               lds.beta[buf][hw][j],
                               !BLOCK_KQ ? 0.f : lane_of(kq, j * StepGeo<D, HW, SPLIT>::LPR), lane);
      if (p.slot_tok) {
        const int slot = __builtin_amdgcn_readfirstlane(lds.tok[buf][j]);
        if (slot >= 0) st.store(p, slot, h);
      }
    }
    if (++blk == w.nb) {
      if (h < w.h1 && w.s_out >= 0) st.store(p, w.s_out, h);
      blk = 0;
      h += HW;
      if (h < w.h1) st.load(p, w.s_in, h);
    }
  }
  __syncthreads();     // the last outputs are in LDS
}

template <typename T> __device__ __forceinline__ void st_raw8(T* p, const Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = r.v[i];
}

// The helper waves; `lane` counts through them.  A conv lane forms 8 channels
// of q, k or one head's v of every token, with the conv's window in
// registers; the lanes behind them form the gate of one token and head each.
template <typename T, int D, int HW, int SPLIT, bool STEP>
__device__ __forceinline__ void step_helper_wave(const StepArgs& p, const StepSpan& w,
                                                 StepLds<D, HW, SPLIT>& lds, int hk, int hv, int lane) {
  typedef StepGeo<D, HW, SPLIT> G;
  constexpr int G8 = D / 8, V8 = G::VC / 8;      // lanes of a q or k row, of a v row
  constexpr int NV = StepLds<D, HW, SPLIT>::NV;
  constexpr int NL = 64 * G::HELPERS, NP = (HW * STEP_TB * V8 + NL - 1) / NL;
  // the step: rows of x on their way, as many as registers allow; each is asked
  // for as soon as the one AHEAD tokens before has served (64 sequences 78.7 us,
  // asked for AHEAD at a time 80.1 us)
  constexpr int AHEAD = HW == 3 && D == 32 ? 1
      : (sizeof(T) == 2 ? 4 : 2) / (HW == 3 || (HW == 2 && sizeof(T) == 4) ? 2 : 1);
  const int C = 2 * hk * D + hv * D;
  // part: 0 q, 1 k, 2 + i v of the round's head i; e: the first of 8 channels
  const int part = SPLIT == 1 || lane < 2 * G8 ? lane / G8 : 2 + (lane - 2 * G8) / V8;
  const int vh = part < 2 ? 0 : part - 2, e = (part < 2 ? lane % G8 : lane % V8) * 8;
  const int gh = (lane - G::CONV_LANES) / STEP_TB, gt = (lane - G::CONV_LANES) % STEP_TB;   // the gate's
  T* out = (T*)p.out;
  // the rule: this lane's tensor and its row stride
  const T* lane_src = STEP ? nullptr : (const T*)p.q;
  int64_t lane_ld = STEP ? 0 : p.ldq;
  if (!STEP && part == 1) { lane_src = (const T*)p.k; lane_ld = p.ldk; }
  if (!STEP && part >= 2) { lane_src = (const T*)p.v; lane_ld = p.ldv; }
  struct Item { int hr, tb; };                   // an item's first head and first token
  float wr[8][4];
  Raw8<T> x3, x2, x1;                            // the window: x[t-3], x[t-2], x[t-1]
  constexpr bool Z_AHEAD = sizeof(T) == 2;       // z's rows a block ahead (registers)
  Raw8<T> z[NP];
  Raw8<T> raw[AHEAD];

  // Row t of x, the lane's 8 channels (past the last token: that one again).
  auto x_row = [&](int ch, int t) __attribute__((always_inline)) {
    return ld_raw8((const T*)p.x + ch + (t < w.t1 ? t : w.t1 - 1) * p.ldx);
  };
  // Requests the rows of x of an item's first tokens.
  auto fetch = [&](const Item& at) __attribute__((always_inline)) {
    if constexpr (STEP) {
      const int h = at.hr + vh;
      if (lane < G::CONV_LANES && (part < 2 || h < w.h1)) {
        const int ch = (part == 0 ? w.kh : part == 1 ? hk + w.kh : 2 * hk + h) * D + e;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) raw[j] = x_row(ch, at.tb + j);
      }
    }
  };
  auto prep = [&](int i, const Item& at) __attribute__((always_inline)) {
    const int buf = i & 1, vb = i % NV, hr = at.hr, tb = at.tb;
    const int nt = w.t1 - tb < STEP_TB ? w.t1 - tb : STEP_TB;
    if (lane < G::CONV_LANES) {
      const int h = hr + vh;
      if (part >= 2 && h >= w.h1) return;
      // the step: this lane's channel of x
      const int ch = (part == 0 ? w.kh : part == 1 ? hk + w.kh : 2 * hk + h) * D + e;
      float* dst = (part == 0 ? lds.q[buf][0] : part == 1 ? lds.k[buf][0] : lds.v[vb][vh][0]) + e;
      const int dst_ld = part < 2 ? D : G::VC;
      if constexpr (STEP) {
        if (tb == w.t0) {
          const T* rows = (const T*)p.cache.conv + (int64_t)w.s_in * p.cache.conv_stride + ch;
          if (w.s_in >= 0) {
            x3 = ld_raw8(rows);
            x2 = ld_raw8(rows + C);
            x1 = ld_raw8(rows + 2 * C);
          } else {
            x3 = x2 = x1 = zero_raw8<T>();
          }
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const float4 a = *reinterpret_cast<const float4*>(p.w_conv + (int64_t)(ch + m) * 4);
            wr[m][0] = a.x; wr[m][1] = a.y; wr[m][2] = a.z; wr[m][3] = a.w;
          }
        }
        // the rows of v's channels have served when their head has; those of
        // q and k are read again in the next round, or by other workgroups
        const bool put_rows = part >= 2 || (w.all && hr + HW >= w.h1);
        auto put = [&](int slot) __attribute__((always_inline)) {
          T* rows = (T*)p.cache.conv + (int64_t)slot * p.cache.conv_stride + ch;
          st_raw8(rows, x3);
          st_raw8(rows + C, x2);
          st_raw8(rows + 2 * C, x1);
        };
        for (int j0 = 0; j0 < nt; j0 += AHEAD) {
#pragma unroll
          for (int j = 0; j < AHEAD; ++j) {
            if (j0 + j < nt) {
              f8 y{};
              auto tap = [&](int i, const f8& xr) __attribute__((always_inline)) {
#pragma unroll
                for (int m = 0; m < 8; ++m) y.v[m] = fmaf(wr[m][i], xr.v[m], y.v[m]);
              };
              tap(0, raw_f8(x3));
              tap(1, raw_f8(x2));
              tap(2, raw_f8(x1));
              tap(3, raw_f8(raw[j]));
              float ss = 0.f;
#pragma unroll
              for (int m = 0; m < 8; ++m) {
                y.v[m] *= sigmoidf_(y.v[m]);
                ss += y.v[m] * y.v[m];
              }
              ss = lane_group_sum<G8>(ss);
              const float r = part >= 2 ? 1.f : rsqrtf(ss + p.l2_eps) * (part == 0 ? p.scale : 1.f);
#pragma unroll
              for (int m = 0; m < 8; ++m) y.v[m] *= r;
              store8(dst + (j0 + j) * dst_ld, y);
              x3 = x2;
              x2 = x1;
              x1 = raw[j];
              if (j0 + AHEAD < nt) raw[j] = x_row(ch, tb + j0 + AHEAD + j);
              if (put_rows && p.slot_tok) {
                const int slot = p.slot_tok[tb + j0 + j];
                if (slot >= 0 && slot < p.cache.n_slots) put(slot);
              }
            }
          }
        }
        if (put_rows && w.s_out >= 0 && tb + nt == w.t1) put(w.s_out);
      } else {
        const float r = part == 0 ? p.scale : 1.f;
        const T* src = lane_src + (part < 2 ? w.kh * D : h * D + w.v0) + e;
        Raw8<T> rows[STEP_TB];                   // rows past the last token: that one again
#pragma unroll
        for (int j = 0; j < STEP_TB; ++j) rows[j] = ld_raw8(src + (tb + j < w.t1 ? tb + j : w.t1 - 1) * lane_ld);
#pragma unroll
        for (int j = 0; j < STEP_TB; ++j)
          if (j < nt) {
            f8 y = raw_f8(rows[j]);
#pragma unroll
            for (int m = 0; m < 8; ++m) y.v[m] *= r;
            store8(dst + j * dst_ld, y);
          }
      }
    } else if (gh < HW && gt < nt && hr + gh < w.h1) {
      const int h = hr + gh;
      const int64_t t = tb + gt;
      if constexpr (STEP) {
        const float xa = to_f(((const T*)p.a)[t * p.lda + h]) + p.dt_bias[h];
        lds.eg[buf][gh][gt] = expf(-expf(p.A_log[h]) * softplus_full(xa));
        lds.beta[buf][gh][gt] = sigmoidf_(to_f(((const T*)p.b)[t * p.ldb + h]));
      } else {
        lds.eg[buf][gh][gt] = expf(p.g[t * hv + h]);
        lds.beta[buf][gh][gt] = p.beta[t * hv + h];
      }
      if (p.slot_tok && gh == 0) {
        const int slot = p.slot_tok[t];
        lds.tok[buf][gt] = slot < p.cache.n_slots ? slot : -1;
      }
    }
  };
  // outputs: lane = (head, token, 8 channels)
  auto each_out = [&](const Item& at, auto&& f) __attribute__((always_inline)) {
    const int tb = at.tb;
#pragma unroll
    for (int s = 0; s < NP; ++s) {
      const int job = (s * NL + lane) / V8, hi = job / STEP_TB, j = job % STEP_TB;
      const int h = at.hr + hi;
      if (hi < HW && h < w.h1 && tb + j < w.t1) f(s, hi, j, (int64_t)(tb + j), h);
    }
  };
  const int oe = lane % V8 * 8;
  f8 wn{};                                       // the norm's 1 + w
  if constexpr (STEP) {
    wn = load8(p.w_norm + oe);
#pragma unroll
    for (int m = 0; m < 8; ++m) wn.v[m] += 1.f;
  }
  auto load_z = [&](const Item& at) __attribute__((always_inline)) {
    if constexpr (STEP && Z_AHEAD)
      each_out(at, [&](int s, int hi, int j, int64_t t, int h) __attribute__((always_inline)) {
        z[s] = ld_raw8((const T*)p.z + t * p.ldz + h * D + oe);
      });
  };
  auto finish = [&](int i, const Item& at) __attribute__((always_inline)) {
    each_out(at, [&](int s, int hi, int j, int64_t t, int h) __attribute__((always_inline)) {
      f8 o = load8(&lds.v[i % NV][hi][j][oe]);
      if constexpr (STEP) {
        float ss = 0.f;
#pragma unroll
        for (int m = 0; m < 8; ++m) ss += o.v[m] * o.v[m];
        ss = lane_group_sum<G8>(ss);
        const float rho = rsqrtf(ss * (1.f / D) + p.norm_eps);
        const f8 zv = Z_AHEAD ? raw_f8(z[s]) : load8((const T*)p.z + t * p.ldz + h * D + oe);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const float sg = sigmoidf_(zv.v[m]);
          o.v[m] *= rho * wn.v[m] * (p.act == 0 ? zv.v[m] * sg : sg);
        }
      }
      store8(out + t * hv * D + h * D + w.v0 + oe, o);
    });
  };

  Item prev{}, cur{}, next{w.h0, w.t0};          // items i - 1, i, i + 1
  fetch(next);
  prep(0, next);
  for (int i = 0; i < w.items; ++i) {
    prev = cur;
    cur = next;
    next.tb += STEP_TB;
    if (next.tb >= w.t1) next = {cur.hr + HW, w.t0};
    __syncthreads();
    if (i + 1 < w.items) fetch(next);
    if (i > 0) finish(i - 1, prev);
    load_z(cur);
    if (i + 1 < w.items) {
      if constexpr (NV == 2) wave_lds_order();   // prep puts v where other lanes read o in finish
      prep(i + 1, next);
    }
  }
  __syncthreads();
  finish(w.items - 1, cur);
}

template <typename T, int D, int HW, int SPLIT, bool STEP, int R>
__global__ void __launch_bounds__((StepGeo<D, HW, SPLIT, R>::THREADS), 4) step_kernel(StepArgs p, int hk, int hv,
                                                                                 int heads, int T_tok) {
  static_assert(SPLIT == 1 || (!STEP && HW == 1), "the norm needs whole rows");
  typedef StepGeo<D, HW, SPLIT, R> G;
  __shared__ StepLds<D, HW, SPLIT> lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int per = hv / heads * SPLIT, n = blockIdx.x / per;
  StepSpan w;
  w.h0 = blockIdx.x % per / SPLIT * heads;
  w.v0 = blockIdx.x % SPLIT * G::VC;
  w.h1 = w.h0 + heads;
  w.kh = w.h0 / (hv / hk);
  w.all = heads == hv / hk;
  token_range(p.cu, n, T_tok, w.t0, w.t1);
  w.s_in = slot_of(p.slot_in, n);
  w.s_out = slot_of(p.slot_out, n);
  if (w.s_in >= p.cache.n_slots || w.s_out >= p.cache.n_slots) {   // a bad slot: NaN rows, no state
    T* out = (T*)p.out;
    const int64_t width = (int64_t)heads * G::VC;
    for (int64_t i = tid; i < (w.t1 - w.t0) * width; i += G::THREADS)
      out[(w.t0 + i / width) * hv * D + (int64_t)w.h0 * D + w.v0 + i % width] = from_f<T>(__builtin_nanf(""));
    return;
  }
  if (w.t0 == w.t1) {   // no tokens: the state passes through
    if (w.s_out < 0 || w.s_out == w.s_in) return;
    if (wave < HW * G::WAVES) {
      StepState<D, SPLIT, R> st(wave % G::WAVES, lane, w.v0);
      for (int h = w.h0 + wave / G::WAVES; h < w.h1; h += HW) {
        st.load(p, w.s_in, h);
        st.store(p, w.s_out, h);
      }
    } else if constexpr (STEP) {
      const int C = 2 * hk * D + hv * D, first = w.all ? 0 : 2, n_grp = (2 - first + heads) * D / 8;
      for (int g = tid - 64 * HW * G::WAVES; g < n_grp * 3; g += 64 * G::HELPERS) {
        const int e = g % n_grp * 8, hd = first + e / D;
        const int64_t ch = (hd == 0 ? w.kh : hd == 1 ? hk + w.kh : 2 * hk + w.h0 + hd - 2) * D + e % D +
                           (int64_t)(g / n_grp) * C;
        store8((T*)p.cache.conv + (int64_t)w.s_out * p.cache.conv_stride + ch,
               w.s_in >= 0 ? load8((const T*)p.cache.conv + (int64_t)w.s_in * p.cache.conv_stride + ch) : f8{});
      }
    }
    return;
  }
  w.nb = (w.t1 - w.t0 - 1) / STEP_TB + 1;
  w.items = (heads + HW - 1) / HW * w.nb;
  if (wave < HW * G::WAVES) step_state_wave<D, HW, SPLIT, !STEP || R == 2, R>(p, w, lds, wave, lane);
  else step_helper_wave<T, D, HW, SPLIT, STEP>(p, w, lds, hk, hv, tid - 64 * HW * G::WAVES);
}

// The conv rows of q's and k's channels, where a key head's value heads were
// in several workgroups and none of them could write what the others read:
// after token t the last three input rows are x[t-2], x[t-1], x[t], reaching
// back into the rows of slot_in.  A thread owns 8 channels of one sequence
// and reads the rows it needs before it writes any.
template <typename T>
__global__ void __launch_bounds__(256) step_rows_kernel(StepArgs p, int n_grp, int C, int T_tok) {
  const int n = blockIdx.y, grp = blockIdx.x * 256 + threadIdx.x;
  if (grp >= n_grp) return;
  int t0, t1;
  token_range(p.cu, n, T_tok, t0, t1);
  const int s_in = slot_of(p.slot_in, n), s_out = slot_of(p.slot_out, n);
  if (s_in >= p.cache.n_slots || s_out >= p.cache.n_slots) return;
  const T* x = (const T*)p.x + grp * 8;
  T* rows = (T*)p.cache.conv + grp * 8;
  Raw8<T> w[3];
#pragma unroll
  for (int j = 0; j < 3; ++j)
    w[j] = s_in >= 0 ? ld_raw8(rows + (int64_t)s_in * p.cache.conv_stride + j * C) : zero_raw8<T>();
  auto put = [&](int slot) {
#pragma unroll
    for (int j = 0; j < 3; ++j) st_raw8(rows + (int64_t)slot * p.cache.conv_stride + j * C, w[j]);
  };
  // without slots for single tokens only the last three rows matter
  for (int t = p.slot_tok || t1 - t0 < 3 ? t0 : t1 - 3; t < t1; ++t) {
    w[0] = w[1];
    w[1] = w[2];
    w[2] = ld_raw8(x + (int64_t)t * p.ldx);
    if (p.slot_tok) {
      const int st = p.slot_tok[t];
      if (st >= 0 && st < p.cache.n_slots) put(st);
    }
  }
  if (s_out >= 0 && (t1 > t0 || s_out != s_in)) put(s_out);
}

template <typename T, int D, int HW, int SPLIT, bool STEP, int R = 4 / SPLIT>
static void launch_step_k(const gdn_shape& s, StepArgs a, int heads, hipStream_t st) {
  constexpr unsigned THREADS = StepGeo<D, HW, SPLIT, R>::THREADS;
  const unsigned per = (unsigned)(s.hv / heads) * SPLIT;
  a.through = (unsigned)s.n_seq * per >= STEP_THROUGH;
  // A launch takes fewer than 2^32 threads; 65535 sequences of 256 heads are
  // more, and go in two.  (With the sequences on a second grid dimension 4 of
  // 1024 tokens take 1045 us instead of 1035 us.)
  const unsigned most = 0xffffffffu / (THREADS * per);
  for (unsigned left = s.n_seq; left > 0;) {
    const unsigned now = left < most ? left : most;
    hipLaunchKernelGGL((step_kernel<T, D, HW, SPLIT, STEP, R>), dim3(now * per), dim3(THREADS), 0, st, a,
                       s.hk, s.hv, heads, (int)s.total_tokens);
    a.cu += now;
    if (a.slot_in) a.slot_in += now;
    if (a.slot_out) a.slot_out += now;
    left -= now;
  }
}

template <typename T, int D, bool STEP>
static void launch_step_d(const gdn_shape& s, const StepArgs& a, hipStream_t st) {
  if constexpr (STEP) {
    const int group = s.hv / s.hk;
    const int64_t groups = (int64_t)s.n_seq * s.hk;
    // While there are no more than 128 groups, heads of a group can go apart,
    // each into a workgroup of its own, at the price of the second launch.
    // Four or more would otherwise take turns two or three at a time (d = 128:
    // 8 sequences of one token, 16 heads over 2: 9.4 us against 21.0 us, of
    // four tokens 11.7 against 29.3 us; 32 over 8: 12.0 against 13.4 us;
    // d = 32: 7.5 against 10.6 us; with 192 groups of four 25.0 against 23.2
    // us).  Two or three go side by side otherwise, so that only pieces of
    // several tokens gain (one sequence, 48 heads over 16: four tokens 10.9
    // against 13.7 us, four sequences 13.2 against 14.6 us, of two 11.3
    // against 10.9 us; 8 heads over 4, eight tokens 14.3 against 15.9 us, four
    // 10.4 both), more heads than CUs later (7 sequences, 48 heads: four 17.1
    // against 16.4 us, eight 23.6 us both), and those of 32 columns never (8
    // tokens: 14.1 against 11.5 us).  The limit of 128 is that of groups of
    // four; larger groups gain most (80 sequences, 16 heads over one: 40
    // against 61 us) and were not measured beyond it.  The lengths are on the
    // device: what counts here are the rows of the call, those of a padded
    // batch among them.
    const bool few = D == 128 && (int64_t)s.n_seq * s.hv <= 256;
    const int64_t pieces = group == 2 ? few ? 8 : 0 : few ? 4 : 8;   // tokens a sequence; 0: never
    const bool apart = groups <= 128 &&
        (group >= 4 || (D == 128 && group > 1 && pieces > 0 && s.total_tokens >= pieces * s.n_seq));
    if (apart) {
      // With a CU to each, a head's rows go over eight waves instead of four (4
      // sequences, 48 heads: 8 tokens 16.7 against 19.1 us, 48 tokens 53.7
      // against 55.9 us; two on a CU have no room for that: 6 sequences, 48
      // tokens 102 against 80 us).
      if (few) launch_step_k<T, D, 1, 1, STEP, D == 128 ? 2 : 4>(s, a, 1, st);
      else launch_step_k<T, D, 1, 1, STEP>(s, a, 1, st);
      const int C = 2 * s.hk * D + s.hv * D, n_grp = 2 * s.hk * D / 8;
      if (a.slot_out || a.slot_tok)
        hipLaunchKernelGGL((step_rows_kernel<T>), dim3((n_grp + 255) / 256, s.n_seq), dim3(256), 0, st, a,
                           n_grp, C, (int)s.total_tokens);
      return;
    }
    // Value heads at a time.  With few workgroups all of a key head's together
    // (one sequence, 48 heads over 16: 9.4 us against 13.6 us one by one; 64
    // sequences 77 against 88 us); with many, one by one in smaller workgroups
    // overlap better (256 sequences 294 against 302 us, 32 heads 198 against
    // 211 us).  They meet at about 2000 workgroups.  Heads of 32 columns have
    // little to overlap and stay together (380 sequences of two tokens, 48
    // heads over 16: three together 49.5 us, two 54.2 us, one by one 56.0 us;
    // 32 heads over 8: two together 33.2 us, four 43.5 us, one by one 42.1 us).
    if (group == 1 || (D == 128 && groups >= 2048)) launch_step_k<T, D, 1, 1, STEP>(s, a, group, st);
    else if (group == 2 || group == 4) launch_step_k<T, D, 2, 1, STEP>(s, a, group, st);
    else launch_step_k<T, D, 3, 1, STEP>(s, a, group, st);
  } else {
    // A head over four workgroups while that still fills the chip's 256 CUs:
    // 8 heads 3.8 us against 4.4 us for one token, 12.4 against 26.4 us for
    // 32; 192 heads 23.3 against 30.7 us; 384 heads 41.1 against 40.3 us.
    if constexpr (D == 128)
      if ((int64_t)s.n_seq * s.hv <= 256) return launch_step_k<T, D, 1, 4, STEP>(s, a, 1, st);
    launch_step_k<T, D, 1, 1, STEP>(s, a, 1, st);
  }
}

template <bool STEP>
static hipError_t launch_step_t(const gdn_shape& s, const StepArgs& a, hipStream_t st) {
  const bool big = s.dk == 128;
  if (s.dtype == GDN_BF16) big ? launch_step_d<bf16, 128, STEP>(s, a, st) : launch_step_d<bf16, 32, STEP>(s, a, st);
  else if (s.dtype == GDN_FP16) big ? launch_step_d<fp16, 128, STEP>(s, a, st) : launch_step_d<fp16, 32, STEP>(s, a, st);
  else big ? launch_step_d<float, 128, STEP>(s, a, st) : launch_step_d<float, 32, STEP>(s, a, st);
  return hipGetLastError();
}

hipError_t launch_recurrent(const gdn_shape& s, const StepArgs& a, hipStream_t st) {
  return launch_step_t<false>(s, a, st);
}

hipError_t launch_step(const gdn_shape& s, const StepArgs& a, hipStream_t st) {
  return launch_step_t<true>(s, a, st);
}

// Check of the slot tables, one workgroup: a table of each slot's writing
// sequence in LDS, for a range of slots at a time.
constexpr int CHECK_RANGE = 8192;
__global__ void __launch_bounds__(256) check_slots_kernel(const int32_t* __restrict__ cu, int n_seq,
                                                          int T_tok, int n_slots,
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
      if (slot_out) claim(slot_out[n], n);
      if (slot_tok) {
        const int t0 = cu[n] < 0 ? 0 : cu[n], t1 = cu[n + 1] < T_tok ? cu[n + 1] : T_tok;
        for (int t = t0; t < t1; ++t) claim(slot_tok[t], n);
      }
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
  hipLaunchKernelGGL(check_slots_kernel, dim3(1), dim3(256), 0, st, cu, s.n_seq, (int)s.total_tokens,
                     n_slots, slot_in, slot_out, slot_tok, out);
  return hipGetLastError();
}

}  // namespace gdn
