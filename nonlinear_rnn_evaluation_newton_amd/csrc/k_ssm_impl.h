// Selective state space scan and its adjoint, per channel d and state n:
//   h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t,  y_t = (C_t h_t + D u_t) silu(z_t)
//
// Layout.  A block holds 64 channels, a wavefront 64 / LPC of them; lane = j * (64 / LPC) + c keeps
// NS states n = j NS .. of channel c in registers and walks time in tiles of
// 16 steps.  B_t and C_t are the same for every channel of a group: lane i of
// each 16-lane row holds them for step i of the tile, and a step's products
// take them by a row broadcast inside the instruction, so they cost neither
// shared memory nor an instruction.  delta and delta u are made once for each
// (step, channel) by the block's threads, 4 channels each, and read back from
// shared memory; the sum over states runs in the lane and then over the LPC
// rows by register swaps, four steps at a time.
#pragma once

#include <utility>

#include "ssm.h"

namespace pr {

template <typename T>
struct Raw4;  // four elements as they are stored
template <>
struct Raw4<uint16_t> {
  uint2 v;
  __device__ float get(int i) const {
    const unsigned w = i < 2 ? v.x : v.y;
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  __device__ void set(const float *f) {
    v.x = (unsigned)f2bf(f[0]) | ((unsigned)f2bf(f[1]) << 16);
    v.y = (unsigned)f2bf(f[2]) | ((unsigned)f2bf(f[3]) << 16);
  }
  __device__ void zero() { v = make_uint2(0, 0); }
  __device__ void one(int i, uint16_t e) {
    unsigned &w = i < 2 ? v.x : v.y;
    w |= (unsigned)e << ((i & 1) * 16);
  }
};
template <>
struct Raw4<float> {
  float4 v;
  __device__ float get(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
  __device__ void set(const float *f) { v = make_float4(f[0], f[1], f[2], f[3]); }
  __device__ void zero() { v = make_float4(0, 0, 0, 0); }
  __device__ void one(int i, float e) { (i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w) = e; }
};

// nv elements at p (0 past them); vec: p is aligned for one load of four
template <typename T>
__device__ inline Raw4<T> load4(const T *p, int nv, bool vec) {
  Raw4<T> r;
  if (vec && nv >= 4) {
    r.v = *reinterpret_cast<const decltype(r.v) *>(p);
  } else {
    r.zero();
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (i < nv) r.one(i, p[i]);
  }
  return r;
}
template <typename T>
__device__ inline void store4(T *p, const float *f, int nv, bool vec) {
  if (vec && nv >= 4) {
    Raw4<T> r;
    r.set(f);
    *reinterpret_cast<decltype(r.v) *>(p) = r.v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (i < nv) stf(p, i, f[i]);
  }
}

// the value that lane I of each 16-lane row holds
template <int I>
__device__ inline float row_bcast(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + I, 0xf, 0xf, true));
}
template <int CTRL>
__device__ inline float dpp_f(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// lower half of the wavefront: a summed over both halves; upper half: b
__device__ inline float half_sums(float a, float b) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// rows 0, 2: a summed over each pair of rows; rows 1, 3: b
__device__ inline float pair_sums(float a, float b) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Sums over the LPC lanes of a channel for LPC steps at once: the lanes of
// group j end with the sum of v[j].
template <int LPC>
__device__ inline float group_sums(const float *v) {
  if constexpr (LPC == 1) return v[0];
  else if constexpr (LPC == 2) return half_sums(v[0], v[1]);
  else return pair_sums(half_sums(v[0], v[2]), half_sums(v[1], v[3]));
}

template <typename F, int... I>
__device__ inline void unrolled(F &&f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
// f(0), f(1), .. f(n - 1), the index a constant of its type
template <int NN, typename F>
__device__ inline void unroll_up(F &&f) {
  unrolled(f, std::make_integer_sequence<int, NN>{});
}

// What a block works on: a channel block of one group, a time segment, a
// sequence.
template <int LPC>
struct Place {
  static constexpr int CW = 64 / LPC, CH = 64, NT = 64 * LPC;  // channels of a wavefront and of a block, threads
  int b, s, cb, g, ch0, nch, t0, t1, len;  // ch0: first channel; nch: channels of the block
  __device__ Place(const SsmArgs &a) {
    const unsigned ncb = (unsigned)(a.G * a.cbg);
    const unsigned i = blockIdx.x;
    cb = (int)(i % ncb);
    const unsigned bs = i / ncb;
    s = (int)(bs % (unsigned)a.S);
    b = (int)(bs / (unsigned)a.S);
    g = cb / a.cbg;
    const int in = (cb - g * a.cbg) * CH;
    ch0 = g * a.dpg + in;
    nch = a.dpg - in < CH ? a.dpg - in : CH;
    t0 = s * a.seglen;
    t1 = a.T - t0 < a.seglen ? a.T : t0 + a.seglen;
    len = seq_len(a.lengths, b, a.T);
  }
};

// NS values n0.. of one step's B or C (0 past N and where the step is not the sequence's)
template <typename T, int NS>
__device__ inline void load_bc(const View &v, const SsmArgs &a, int b, int t, bool on, int g, int n0, float *o) {
  const T *p = reinterpret_cast<const T *>(v.p) + b * v.sb + t * v.st + (long long)g * a.N + n0;
#pragma unroll
  for (int q = 0; q < NS; q += 4) {
    const int left = on ? a.N - n0 - q : 0;
    const Raw4<T> r = load4<T>(p + q, left, a.vecn != 0);
#pragma unroll
    for (int i = 0; i < 4; i++) o[q + i] = r.get(i);
  }
}

template <int NS>
__device__ inline void load_state(const float *p, int n0, int N, bool on, float *h) {
#pragma unroll
  for (int q = 0; q < NS; q += 4) {
    const int left = on ? N - n0 - q : 0;
    if (left >= 4 && (N & 3) == 0) {
      const float4 v = *reinterpret_cast<const float4 *>(p + n0 + q);
      h[q] = v.x; h[q + 1] = v.y; h[q + 2] = v.z; h[q + 3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) h[q + i] = i < left ? p[n0 + q + i] : 0.f;
    }
  }
}
template <int NS>
__device__ inline void store_state(float *p, int n0, int N, bool on, const float *h) {
#pragma unroll
  for (int q = 0; q < NS; q += 4) {
    const int left = on ? N - n0 - q : 0;
    if (left >= 4 && (N & 3) == 0) {
      *reinterpret_cast<float4 *>(p + n0 + q) = make_float4(h[q], h[q + 1], h[q + 2], h[q + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (i < left) p[n0 + q + i] = h[q + i];
    }
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// FULL: outputs, from the state that enters the segment (a.agg where S > 1,
// else h0).  Not FULL: the segment's end state from zero and its sum of delta.
template <typename T, int NS, int LPC, bool FULL>
__global__ __launch_bounds__(64 * LPC) void k_ssm_fwd(SsmArgs a) {
  using P = Place<LPC>;
  constexpr int CW = P::CW, CH = P::CH, NT = P::NT, TL = SSM_TL, UPT = TL * CH / 4 / NT, YS = CH + 16;
  __shared__ float2 sdx[2][TL][CH];
  __shared__ float sy[FULL ? 2 : 1][FULL ? TL : 1][YS];
  const P w(a);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int j = lane / CW, c = wave * CW + lane % CW, n0 = j * NS;
  const bool on = c < w.nch;
  const int d = w.ch0 + c;
  const int end = w.t1 < w.len ? w.t1 : w.len;  // steps past it leave the state as it is
  const int ntiles = end > w.t0 ? (end - w.t0 + TL - 1) / TL : 0;
  const long long dn = (long long)a.D * a.N;

  float A2[NS], h[NS];
  load_state<NS>(a.A + (long long)(on ? d : 0) * a.N, n0, a.N, on, A2);
#pragma unroll
  for (int k = 0; k < NS; k++) A2[k] *= 1.4426950408889634f;
  if constexpr (FULL) {
    const float *hp = a.S > 1 ? a.agg + ((long long)w.b * a.S + w.s) * dn : a.h0 ? a.h0 + w.b * dn : nullptr;
    load_state<NS>(hp + (long long)d * a.N, n0, a.N, on && hp, h);
  } else {
#pragma unroll
    for (int k = 0; k < NS; k++) h[k] = 0.f;
  }
  float dsum = 0.f;

  // staging: unit q of a thread is 4 channels of one step of the tile
  int ur[UPT], uc[UPT], unv[UPT];
  float ub[UPT][4], uD[UPT][4];
#pragma unroll
  for (int q = 0; q < UPT; q++) {
    const int id = q * NT + tid;
    ur[q] = id / (CH / 4);
    uc[q] = (id % (CH / 4)) * 4;
    unv[q] = w.nch - uc[q];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const bool in = i < unv[q];
      ub[q][i] = in && a.bias ? a.bias[w.ch0 + uc[q] + i] : 0.f;
      uD[q][i] = FULL && in && a.Dk ? a.Dk[w.ch0 + uc[q] + i] : 0.f;
    }
  }
  Raw4<T> ru[UPT], rd[UPT], rz[UPT], pu[UPT], pz[UPT];
  float nB[NS], nC[NS];
  const bool vec = a.vec != 0;
  auto load_tile = [&](int t0) {
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const int t = t0 + ur[q], nv = t < end ? unv[q] : 0;
      ru[q] = load4<T>((const T *)a.u.p + w.b * a.u.sb + t * a.u.st + w.ch0 + uc[q], nv, vec);
      rd[q] = load4<T>((const T *)a.dt.p + w.b * a.dt.sb + t * a.dt.st + w.ch0 + uc[q], nv, vec);
      if (FULL && a.z.p) rz[q] = load4<T>((const T *)a.z.p + w.b * a.z.sb + t * a.z.st + w.ch0 + uc[q], nv, vec);
    }
    const int t = t0 + (lane & 15);
    load_bc<T, NS>(a.Bm, a, w.b, t, t < end, w.g, n0, nB);
    if (FULL) load_bc<T, NS>(a.Cm, a, w.b, t, t < end, w.g, n0, nC);
  };
  auto output = [&](int tile) {
    if constexpr (FULL) {
      const int t0 = w.t0 + tile * TL;
#pragma unroll
      for (int q = 0; q < UPT; q++) {
        const int t = t0 + ur[q];
        if (t < w.t1 && unv[q] > 0) {
          float o[4];
          const bool live = t < end;
#pragma unroll
          for (int i = 0; i < 4; i++) {
            float v = fmaf(uD[q][i], pu[q].get(i), sy[tile & 1][ur[q]][uc[q] + i]);
            if (a.z.p) {
              const float zz = pz[q].get(i);
              v *= zz * fsigm(zz);
            }
            o[i] = live ? v : 0.f;
          }
          store4<T>((T *)a.y.p + w.b * a.y.sb + t * a.y.st + w.ch0 + uc[q], o, unv[q], vec);
        }
      }
    }
  };

  if (ntiles > 0) load_tile(w.t0);
  for (int tile = 0; tile < ntiles; tile++) {
    const int t0 = w.t0 + tile * TL, p = tile & 1;
    float B[NS], C[NS];
#pragma unroll
    for (int k = 0; k < NS; k++) {
      B[k] = nB[k];
      if (FULL) C[k] = nC[k];
    }
    Raw4<T> cu[UPT], cz[UPT];
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const bool live = t0 + ur[q] < end;
      float dx[8];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float v = rd[q].get(i) + ub[q][i];
        if (a.softplus) v = softplus_f(v);
        v = live && i < unv[q] ? v : 0.f;
        dx[2 * i] = v;
        dx[2 * i + 1] = v * ru[q].get(i);
      }
      float4 *o = reinterpret_cast<float4 *>(&sdx[p][ur[q]][uc[q]]);
      o[0] = make_float4(dx[0], dx[1], dx[2], dx[3]);
      o[1] = make_float4(dx[4], dx[5], dx[6], dx[7]);
      cu[q] = ru[q];
      cz[q] = rz[q];
    }
    if (tile + 1 < ntiles) load_tile(t0 + TL);
    lds_barrier();
    if (tile > 0) output(tile - 1);
    if constexpr (FULL) {
      if (a.states) {
        const int nt = (a.T + TL - 1) / TL;
        store_state<NS>(a.states + ((long long)w.b * nt + t0 / TL) * dn + (long long)d * a.N, n0, a.N, on, h);
      }
    }
    unroll_up<TL / 4>([&](auto quad) {
      constexpr int I0 = decltype(quad)::value * 4;
      float acc[4];
      unroll_up<4>([&](auto within) {
        constexpr int W = decltype(within)::value, I = I0 + W;
        const float2 dx = sdx[p][I][c];
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NS; k++) {
          const float e = __builtin_amdgcn_exp2f(dx.x * A2[k]);
          h[k] = fmaf(e, h[k], row_bcast<I>(B[k]) * dx.y);
          if (FULL) s = fmaf(row_bcast<I>(C[k]), h[k], s);
        }
        if (!FULL) dsum += dx.x;
        acc[W] = s;
      });
      if constexpr (FULL) {
#pragma unroll
        for (int q = 0; q < 4; q += LPC) sy[p][I0 + q + j][c] = group_sums<LPC>(acc + q);
      }
    });
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      pu[q] = cu[q];
      pz[q] = cz[q];
    }
  }
  if constexpr (FULL) {
    if (ntiles > 0) {
      lds_barrier();
      output(ntiles - 1);
    }
    // steps past the sequence's length
    const int z0 = w.t0 + ntiles * TL;
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t = z0; t < w.t1; t += TL)
#pragma unroll
      for (int q = 0; q < UPT; q++)
        if (t + ur[q] < w.t1 && unv[q] > 0)
          store4<T>((T *)a.y.p + w.b * a.y.sb + (t + ur[q]) * a.y.st + w.ch0 + uc[q], zero, unv[q], vec);
    const int last = w.len > 0 ? (w.len - 1) / a.seglen : 0;
    if (a.hlast && w.s == last)
      store_state<NS>(a.hlast + w.b * dn + (long long)d * a.N, n0, a.N, on, h);
  } else {
    const long long at = (long long)w.b * a.S + w.s;
    store_state<NS>(a.agg + at * dn + (long long)d * a.N, n0, a.N, on, h);
    if (j == 0 && on) a.sumd[at * a.D + d] = dsum;
  }
}

// ---------------------------------------------------------------------------
// adjoint
// ---------------------------------------------------------------------------
// With e_t = dy_t silu(z_t), the adjoint state g_t = C_t e_t + a_{t+1} g_{t+1}
// runs backwards; r_t = a_t g_t is what a step hands to the one before it.
// Not FULL: the segment's r at its first step from zero behind it.
template <typename T, int NS, int LPC>
__global__ __launch_bounds__(64 * LPC) void k_ssm_adj_agg(SsmArgs a) {
  using P = Place<LPC>;
  constexpr int CW = P::CW, CH = P::CH, NT = P::NT, TL = SSM_TL, UPT = TL * CH / 4 / NT;
  __shared__ float2 sde[2][TL][CH];  // delta, e
  const P w(a);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int j = lane / CW, c = wave * CW + lane % CW, n0 = j * NS;
  const bool on = c < w.nch, vec = a.vec != 0;
  const int d = w.ch0 + c;
  const int end = w.t1 < w.len ? w.t1 : w.len;
  const int ntiles = end > w.t0 ? (end - w.t0 + TL - 1) / TL : 0;
  const long long dn = (long long)a.D * a.N;
  float A2[NS], r[NS];
  load_state<NS>(a.A + (long long)(on ? d : 0) * a.N, n0, a.N, on, A2);
#pragma unroll
  for (int k = 0; k < NS; k++) {
    A2[k] *= 1.4426950408889634f;
    r[k] = 0.f;
  }
  float dsum = 0.f;
  for (int tile = ntiles - 1; tile >= 0; tile--) {
    const int t0 = w.t0 + tile * TL, p = tile & 1;
    float C[NS];
    const int tb = t0 + (lane & 15);
    load_bc<T, NS>(a.Cm, a, w.b, tb, tb < end, w.g, n0, C);
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const int id = q * NT + tid, row = id / (CH / 4), cc = (id % (CH / 4)) * 4, t = t0 + row;
      const int nv = t < end ? w.nch - cc : 0;
      const long long off = w.ch0 + cc;
      const Raw4<T> rd = load4<T>((const T *)a.dt.p + w.b * a.dt.sb + t * a.dt.st + off, nv, vec);
      const Raw4<T> ry = load4<T>((const T *)a.dy.p + w.b * a.dy.sb + t * a.dy.st + off, nv, vec);
      Raw4<T> rz;
      if (a.z.p) rz = load4<T>((const T *)a.z.p + w.b * a.z.sb + t * a.z.st + off, nv, vec);
      float o[8];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const bool in = i < nv;
        float v = rd.get(i) + (in && a.bias ? a.bias[off + i] : 0.f);
        if (a.softplus) v = softplus_f(v);
        float e = ry.get(i);
        if (a.z.p) {
          const float zz = rz.get(i);
          e *= zz * fsigm(zz);
        }
        o[2 * i] = in ? v : 0.f;
        o[2 * i + 1] = in ? e : 0.f;
      }
      float4 *q4 = reinterpret_cast<float4 *>(&sde[p][row][cc]);
      q4[0] = make_float4(o[0], o[1], o[2], o[3]);
      q4[1] = make_float4(o[4], o[5], o[6], o[7]);
    }
    lds_barrier();
    unroll_up<TL>([&](auto ic) {
      constexpr int I = TL - 1 - decltype(ic)::value;
      const float2 de = sde[p][I][c];
#pragma unroll
      for (int k = 0; k < NS; k++) {
        const float e = __builtin_amdgcn_exp2f(de.x * A2[k]);
        r[k] = e * fmaf(row_bcast<I>(C[k]), de.y, r[k]);
      }
      dsum += de.x;
    });
  }
  const long long at = (long long)w.b * a.S + w.s;
  store_state<NS>(a.agg + at * dn + (long long)d * a.N, n0, a.N, on, r);
  if (j == 0 && on) a.sumd[at * a.D + d] = dsum;
}

// The gradients of one segment, 4 states per lane and group of states (NG
// groups of 4 LPC states one after the other).  Per tile the states of its 16
// steps are made again from the saved one that enters it and stay in
// registers with their decays for the walk back.
template <typename T, int NG, int LPC>
__global__ __launch_bounds__(64 * LPC) void k_ssm_adj(SsmArgs a) {
  using P = Place<LPC>;
  constexpr int CW = P::CW, CH = P::CH, NT = P::NT, TL = SSM_TL, UPT = TL * CH / 4 / NT, YS = CH + 16;
  constexpr int GP = 4 * LPC, NP = NG * GP;  // states of a group, padded number of states
  struct Buf {
    float2 dx[TL][CH];                      // delta, delta u
    float e[TL][CH];
    float sum[3][TL][YS];                   // sums over states: C h, B g, A r h_{t-1}
    float bc[LPC][TL][2 * NP];              // each wave's dB | dC
  };
  __shared__ Buf buf[2];
  const P w(a);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int j = lane / CW, c = wave * CW + lane % CW;
  const bool on = c < w.nch, vec = a.vec != 0, gate = a.z.p != nullptr;
  const int d = w.ch0 + c;
  const int end = w.t1 < w.len ? w.t1 : w.len;
  const int ntiles = end > w.t0 ? (end - w.t0 + TL - 1) / TL : 0;
  const int nt = (a.T + TL - 1) / TL;
  const long long dn = (long long)a.D * a.N;
  const long long at = (long long)w.b * a.S + w.s;

  float A[NG][4], r[NG][4], dA[NG][4];
#pragma unroll
  for (int g = 0; g < NG; g++) {
    const int n0 = g * GP + j * 4;
    load_state<4>(a.A + (long long)(on ? d : 0) * a.N, n0, a.N, on, A[g]);
    const float *rp = a.S > 1 ? a.agg + at * dn : a.dhlast ? a.dhlast + w.b * dn : nullptr;
    load_state<4>(rp + (long long)d * a.N, n0, a.N, on && rp, r[g]);
#pragma unroll
    for (int k = 0; k < 4; k++) dA[g][k] = 0.f;
  }

  int ur[UPT], uc[UPT], unv[UPT];
  float ub[UPT][4], uD[UPT][4], accD[UPT][4], accb[UPT][4];
#pragma unroll
  for (int q = 0; q < UPT; q++) {
    const int id = q * NT + tid;
    ur[q] = id / (CH / 4);
    uc[q] = (id % (CH / 4)) * 4;
    unv[q] = w.nch - uc[q];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const bool in = i < unv[q];
      ub[q][i] = in && a.bias ? a.bias[w.ch0 + uc[q] + i] : 0.f;
      uD[q][i] = in && a.Dk ? a.Dk[w.ch0 + uc[q] + i] : 0.f;
      accD[q][i] = accb[q][i] = 0.f;
    }
  }
  struct Raws {
    Raw4<T> u[UPT], d[UPT], y[UPT], z[UPT];
  };
  Raws nx, cur, pv;
  // delta and e of the tile that `output` finishes: its buffer may be refilled meanwhile
  float cdl[UPT][4], ce[UPT][4], pdl[UPT][4], pe[UPT][4];
  float nB[NG][4], nC[NG][4], nh[NG][4];
  auto load_tile = [&](int tile) {
    const int t0 = w.t0 + tile * TL;
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const int t = t0 + ur[q], nv = t < end ? unv[q] : 0;
      const long long off = w.ch0 + uc[q];
      nx.u[q] = load4<T>((const T *)a.u.p + w.b * a.u.sb + t * a.u.st + off, nv, vec);
      nx.d[q] = load4<T>((const T *)a.dt.p + w.b * a.dt.sb + t * a.dt.st + off, nv, vec);
      nx.y[q] = load4<T>((const T *)a.dy.p + w.b * a.dy.sb + t * a.dy.st + off, nv, vec);
      if (gate) nx.z[q] = load4<T>((const T *)a.z.p + w.b * a.z.sb + t * a.z.st + off, nv, vec);
    }
    const int t = t0 + (lane & 15);
#pragma unroll
    for (int g = 0; g < NG; g++) {
      const int n0 = g * GP + j * 4;
      load_bc<T, 4>(a.Bm, a, w.b, t, t < end, w.g, n0, nB[g]);
      load_bc<T, 4>(a.Cm, a, w.b, t, t < end, w.g, n0, nC[g]);
      load_state<4>(a.states + ((long long)w.b * nt + t0 / TL) * dn + (long long)d * a.N, n0, a.N, on, nh[g]);
    }
  };
  // gradients of a finished tile from its sums
  auto output = [&](int tile) {
    const int t0 = w.t0 + tile * TL;
    const Buf &f = buf[tile & 1];
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const int t = t0 + ur[q];
      if (t < w.t1 && unv[q] > 0) {
        const bool live = t < end;
        float du[4], ddt[4], dz[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int cc = uc[q] + i;
          const float u = pv.u[q].get(i), v = pv.d[q].get(i) + ub[q][i];
          const float e = pe[q][i], gb = f.sum[1][ur[q]][cc];
          du[i] = fmaf(pdl[q][i], gb, uD[q][i] * e);
          float dd = fmaf(u, gb, f.sum[2][ur[q]][cc]);
          if (a.softplus) dd *= fsigm(v);
          ddt[i] = dd;
          if (gate) {
            const float zz = pv.z[q].get(i), s = fsigm(zz);
            const float y0 = fmaf(uD[q][i], u, f.sum[0][ur[q]][cc]);
            dz[i] = live ? pv.y[q].get(i) * y0 * (s * fmaf(zz, 1.f - s, 1.f)) : 0.f;
          }
          if (!live) du[i] = ddt[i] = 0.f;
          if (live && i < unv[q]) {
            accD[q][i] = fmaf(e, u, accD[q][i]);
            accb[q][i] += ddt[i];
          }
        }
        const long long off = w.ch0 + uc[q];
        if (a.du.p) store4<T>((T *)a.du.p + w.b * a.du.sb + t * a.du.st + off, du, unv[q], vec);
        if (a.ddt.p) store4<T>((T *)a.ddt.p + w.b * a.ddt.sb + t * a.ddt.st + off, ddt, unv[q], vec);
        if (gate && a.dz.p) store4<T>((T *)a.dz.p + w.b * a.dz.sb + t * a.dz.st + off, dz, unv[q], vec);
      }
    }
    // the waves' dB | dC of each step, to this channel block's partial
    for (int i = tid; i < TL * 2 * NP; i += NT) {
      const int row = i / (2 * NP), n = i % (2 * NP), t = t0 + row;
      if (t < end) {
        float v = f.bc[0][row][n];
#pragma unroll
        for (int m = 1; m < LPC; m++) v += f.bc[m][row][n];
        const int in = w.cb - w.g * a.cbg;
        a.part[((((long long)in * a.B + w.b) * a.T + t) * a.G + w.g) * (2 * NP) + n] = v;
      }
    }
  };

  if (ntiles > 0) load_tile(ntiles - 1);
  for (int tile = ntiles - 1; tile >= 0; tile--) {
    const int t0 = w.t0 + tile * TL;
    Buf &f = buf[tile & 1];
    float B[NG][4], C[NG][4], hin[NG][4];
#pragma unroll
    for (int g = 0; g < NG; g++)
#pragma unroll
      for (int k = 0; k < 4; k++) {
        B[g][k] = nB[g][k];
        C[g][k] = nC[g][k];
        hin[g][k] = nh[g][k];
      }
    cur = nx;
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const bool live = t0 + ur[q] < end;
      float dx[8], ee[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float v = cur.d[q].get(i) + ub[q][i];
        if (a.softplus) v = softplus_f(v);
        float e = cur.y[q].get(i);
        if (gate) {
          const float zz = cur.z[q].get(i);
          e *= zz * fsigm(zz);
        }
        const bool in = live && i < unv[q];
        v = in ? v : 0.f;
        dx[2 * i] = v;
        dx[2 * i + 1] = v * cur.u[q].get(i);
        ee[i] = in ? e : 0.f;
        cdl[q][i] = v;
        ce[q][i] = ee[i];
      }
      float4 *o = reinterpret_cast<float4 *>(&f.dx[ur[q]][uc[q]]);
      o[0] = make_float4(dx[0], dx[1], dx[2], dx[3]);
      o[1] = make_float4(dx[4], dx[5], dx[6], dx[7]);
      *reinterpret_cast<float4 *>(&f.e[ur[q]][uc[q]]) = make_float4(ee[0], ee[1], ee[2], ee[3]);
    }
    if (tile > 0) load_tile(tile - 1);
    lds_barrier();
    if (tile + 1 < ntiles) output(tile + 1);
#pragma unroll
    for (int g = 0; g < NG; g++) {
      float hs[TL][4], as[TL][4];
      float A2[4];
#pragma unroll
      for (int k = 0; k < 4; k++) A2[k] = A[g][k] * 1.4426950408889634f;
      unroll_up<TL>([&](auto ic) {
        constexpr int I = decltype(ic)::value;
        const float2 dx = f.dx[I][c];
#pragma unroll
        for (int k = 0; k < 4; k++) {
          as[I][k] = __builtin_amdgcn_exp2f(dx.x * A2[k]);
          const float before = I > 0 ? hs[I > 0 ? I - 1 : 0][k] : hin[g][k];
          hs[I][k] = fmaf(as[I][k], before, row_bcast<I>(B[g][k]) * dx.y);
        }
        // keeps the compiler from spreading the steps' temporaries over the whole tile
        if constexpr (I % 4 == 3) __builtin_amdgcn_sched_barrier(0);
      });
      float sums[3][4];  // of four steps, over the lane's states
      unroll_up<TL>([&](auto ic) {
        constexpr int I = TL - 1 - decltype(ic)::value;
        const float2 dx = f.dx[I][c];
        const float e = f.e[I][c];
        float y0 = 0.f, gb = 0.f, qa = 0.f;
        float db[4], dc[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const float before = I > 0 ? hs[I > 0 ? I - 1 : 0][k] : hin[g][k];
          const float gg = fmaf(row_bcast<I>(C[g][k]), e, r[g][k]);
          y0 = fmaf(row_bcast<I>(C[g][k]), hs[I][k], y0);
          gb = fmaf(row_bcast<I>(B[g][k]), gg, gb);
          db[k] = dx.y * gg;
          dc[k] = e * hs[I][k];
          r[g][k] = as[I][k] * gg;
          const float q = r[g][k] * before;
          qa = fmaf(A[g][k], q, qa);
          dA[g][k] = fmaf(dx.x, q, dA[g][k]);
        }
        sums[0][I % 4] = y0;
        sums[1][I % 4] = gb;
        sums[2][I % 4] = qa;
        // over the channels of each row
#pragma unroll
        for (int k = 0; k < 4; k++) {
          db[k] += dpp_f<0x128>(db[k]);  // row_ror:8, 4, 2, 1
          dc[k] += dpp_f<0x128>(dc[k]);
          db[k] += dpp_f<0x124>(db[k]);
          dc[k] += dpp_f<0x124>(dc[k]);
          db[k] += dpp_f<0x122>(db[k]);
          dc[k] += dpp_f<0x122>(dc[k]);
          db[k] += dpp_f<0x121>(db[k]);
          dc[k] += dpp_f<0x121>(dc[k]);
        }
        if constexpr (LPC < 4) {  // rows that hold other channels of the same states
#pragma unroll
          for (int k = 0; k < 4; k++) {
            db[k] += __shfl_xor(db[k], 16, 64);
            dc[k] += __shfl_xor(dc[k], 16, 64);
            if constexpr (LPC == 1) {
              db[k] += __shfl_xor(db[k], 32, 64);
              dc[k] += __shfl_xor(dc[k], 32, 64);
            }
          }
        }
        if (lane % CW == 0) {
          float *o = &f.bc[wave][I][g * GP + j * 4];
          *reinterpret_cast<float4 *>(o) = make_float4(db[0], db[1], db[2], db[3]);
          *reinterpret_cast<float4 *>(o + NP) = make_float4(dc[0], dc[1], dc[2], dc[3]);
        }
        if constexpr (I % 4 == 0) {
#pragma unroll
          for (int m = 0; m < 3; m++)
#pragma unroll
            for (int q = 0; q < 4; q += LPC) {
              float &o = f.sum[m][I + q + j][c];  // the same lane adds each group's part
              const float v = group_sums<LPC>(sums[m] + q);
              o = g > 0 ? o + v : v;
            }
          __builtin_amdgcn_sched_barrier(0);
        }
      });
    }
    pv = cur;
#pragma unroll
    for (int q = 0; q < UPT; q++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        pdl[q][i] = cdl[q][i];
        pe[q][i] = ce[q][i];
      }
  }
  if (ntiles > 0) {
    lds_barrier();
    output(0);
  }
  // steps past the length: zero gradients
  const float zero[4] = {0.f, 0.f, 0.f, 0.f};
  for (int t = w.t0 + ntiles * TL; t < w.t1; t += TL)
#pragma unroll
    for (int q = 0; q < UPT; q++)
      if (t + ur[q] < w.t1 && unv[q] > 0) {
        const long long off = w.ch0 + uc[q];
        const int tt = t + ur[q];
        if (a.du.p) store4<T>((T *)a.du.p + w.b * a.du.sb + tt * a.du.st + off, zero, unv[q], vec);
        if (a.ddt.p) store4<T>((T *)a.ddt.p + w.b * a.ddt.sb + tt * a.ddt.st + off, zero, unv[q], vec);
        if (gate && a.dz.p) store4<T>((T *)a.dz.p + w.b * a.dz.sb + tt * a.dz.st + off, zero, unv[q], vec);
      }
#pragma unroll
  for (int g = 0; g < NG; g++) {
    const int n0 = g * GP + j * 4;
    store_state<4>(a.pA + at * dn + (long long)d * a.N, n0, a.N, on, dA[g]);
    if (a.dh0 && w.s == 0) store_state<4>(a.dh0 + w.b * dn + (long long)d * a.N, n0, a.N, on, r[g]);
  }
  // dD and the bias' gradient: over the tile's rows, which different threads hold
  __syncthreads();
  float *red = reinterpret_cast<float *>(&buf[0]);  // [2][TL][CH]
#pragma unroll
  for (int q = 0; q < UPT; q++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      red[ur[q] * CH + uc[q] + i] = accD[q][i];
      red[(TL + ur[q]) * CH + uc[q] + i] = accb[q][i];
    }
  __syncthreads();
  for (int i = tid; i < 2 * CH; i += NT) {
    const int m = i / CH, cc = i % CH;
    if (cc < w.nch) {
      float v = 0.f;
#pragma unroll
      for (int row = 0; row < TL; row++) v += red[(m * TL + row) * CH + cc];
      a.pD[(at * 2 + m) * a.D + w.ch0 + cc] = v;
    }
  }
}

// ---------------------------------------------------------------------------
template <typename T, int NS, int LPC>
hipError_t ssm_launch_geom(const SsmArgs &a, int what, hipStream_t s) {
  const dim3 grid((unsigned)((long long)a.B * a.S * a.G * a.cbg));
  switch (what) {
    case SSM_FWD: k_ssm_fwd<T, NS, LPC, true><<<grid, 64 * LPC, 0, s>>>(a); break;
    case SSM_FWD_AGG: k_ssm_fwd<T, NS, LPC, false><<<grid, 64 * LPC, 0, s>>>(a); break;
    case SSM_ADJ: k_ssm_adj<T, NS / 4, LPC><<<grid, 64 * LPC, 0, s>>>(a); break;
    default: k_ssm_adj_agg<T, NS, LPC><<<grid, 64 * LPC, 0, s>>>(a); break;
  }
  return hipGetLastError();
}

template <typename T>
hipError_t ssm_launch(const SsmArgs &a, int what, hipStream_t s) {
  const SsmGeom g = ssm_geom(a.N);
  if (g.ns == 4 && g.lpc == 1) return ssm_launch_geom<T, 4, 1>(a, what, s);
  if (g.ns == 4 && g.lpc == 2) return ssm_launch_geom<T, 4, 2>(a, what, s);
  if (g.ns == 4) return ssm_launch_geom<T, 4, 4>(a, what, s);
  if (g.ns == 8) return ssm_launch_geom<T, 8, 4>(a, what, s);
  return ssm_launch_geom<T, 16, 4>(a, what, s);
}

}  // namespace pr
