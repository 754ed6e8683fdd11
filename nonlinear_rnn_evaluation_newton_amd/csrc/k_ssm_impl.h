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

// the tile bodies are large and called from several places of an unrolled loop:
// out of line, their captures would go to memory
#define PR_INLINE __attribute__((always_inline))

namespace pr {

// Loads and stores in the tile loops are buffer instructions whose range check
// drops what is outside (a load gives 0): none sits under a branch, so the
// compiler's count of accesses in flight stays exact and a wait for one tile's
// data leaves the later tiles' loads and the recent stores in flight.
typedef __amdgpu_buffer_rsrc_t SRsrc;
typedef unsigned su32x2 __attribute__((ext_vector_type(2)));
typedef unsigned su32x4 __attribute__((ext_vector_type(4)));
constexpr unsigned S_OOB = 0x80000000u;  // outside every resource
__device__ inline SRsrc s_rsrc(const void *base, bool on = true) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, on ? 0x7fffffff : 0, 0x00020000);
}

template <typename T>
struct Raw4;  // four elements as they are stored
template <>
struct Raw4<uint16_t> {
  su32x2 v;
  __device__ float get(int i) const {
    const unsigned w = i < 2 ? v.x : v.y;
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  __device__ void set(const float *f) {
    v.x = (unsigned)f2bf(f[0]) | ((unsigned)f2bf(f[1]) << 16);
    v.y = (unsigned)f2bf(f[2]) | ((unsigned)f2bf(f[3]) << 16);
  }
};
template <>
struct Raw4<float> {
  su32x4 v;
  __device__ float get(int i) const { return __uint_as_float(v[i]); }
  __device__ void set(const float *f) {
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = __float_as_uint(f[i]);
  }
};

// nv elements (at most four) from byte `off` on, 0 past them.  VEC: one
// access, nv is 4 or not positive; else element by element.
template <typename T, bool VEC>
__device__ inline Raw4<T> load4(SRsrc r, unsigned off, int nv) {
  Raw4<T> o;
  if constexpr (VEC) {
    const unsigned at = nv > 0 ? off : S_OOB;
    if constexpr (sizeof(T) == 2) o.v = __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
    else o.v = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
  } else if constexpr (sizeof(T) == 2) {
    unsigned e[4];
#pragma unroll
    for (int i = 0; i < 4; i++) e[i] = __builtin_amdgcn_raw_buffer_load_b16(r, i < nv ? off + 2 * i : S_OOB, 0, 0);
    o.v.x = e[0] | (e[1] << 16);
    o.v.y = e[2] | (e[3] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) o.v[i] = __builtin_amdgcn_raw_buffer_load_b32(r, i < nv ? off + 4 * i : S_OOB, 0, 0);
  }
  return o;
}
template <typename T, bool VEC>
__device__ inline void store4(SRsrc r, unsigned off, const float *f, int nv) {
  Raw4<T> o;
  o.set(f);
  if constexpr (VEC) {
    const unsigned at = nv > 0 ? off : S_OOB;
    if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b64(o.v, r, at, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b128(o.v, r, at, 0, 0);
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; i++)
      __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(o.v[i >> 1] >> (16 * (i & 1))), r, i < nv ? off + 2 * i : S_OOB,
                                            0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      __builtin_amdgcn_raw_buffer_store_b32(o.v[i], r, i < nv ? off + 4 * i : S_OOB, 0, 0);
  }
}

// the resource of steps t.. of sequence b of an array
template <typename T>
__device__ inline SRsrc rows_of(const View &v, int b, int t) {
  return s_rsrc((const T *)v.p + b * v.sb + t * v.st, v.p != nullptr);
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

// Fused multiply-adds whose second factor is broadcast from a lane of each row
// inside the instruction (the compiler keeps such a broadcast apart).  A value
// that a vector instruction wrote may be broadcast from the third instruction
// after it on; what stands before these is the compiler's choice, so each group
// of four waits for that itself.
// acc[w] += v[w] times c of lane I0 + w
template <int I0>
__device__ inline void fma_bcast_steps(float *acc, float c, float v0, float v1, float v2, float v3) {
  asm("s_nop 1\n\t"
      "v_fmac_f32_dpp %0, %4, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %1, %4, %6 row_newbcast:%10 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %2, %4, %7 row_newbcast:%11 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %3, %4, %8 row_newbcast:%12 row_mask:0xf bank_mask:0xf"
      : "+v"(acc[0]), "+v"(acc[1]), "+v"(acc[2]), "+v"(acc[3])
      : "v"(c), "v"(v0), "v"(v1), "v"(v2), "v"(v3), "n"(I0), "n"(I0 + 1), "n"(I0 + 2), "n"(I0 + 3));
}
// acc[k] += v times c[k] of lane I
template <int I>
__device__ inline void fma_bcast_states(float *acc, const float *c, float v) {
  asm("s_nop 1\n\t"
      "v_fmac_f32_dpp %0, %4, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %1, %5, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %2, %6, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %3, %7, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
      : "+v"(acc[0]), "+v"(acc[1]), "+v"(acc[2]), "+v"(acc[3])
      : "v"(c[0]), "v"(c[1]), "v"(c[2]), "v"(c[3]), "v"(v), "n"(I));
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

// acc[w] = sum over k of v[w][k] times the value of cf[k] that lane I0 + w of
// each row holds.  The sum ends in a plain addition: the register swaps that
// use it need wait states that the compiler counts from instructions it knows.
template <int I0, int NS>
__device__ inline void sum_bcast(float *acc, const float *cf, const float (*v)[NS]) {
  float first[4];
  unroll_up<4>([&](auto within) PR_INLINE {
    constexpr int W = decltype(within)::value;
    first[W] = row_bcast<I0 + W>(cf[0]) * v[W][0];
    acc[W] = row_bcast<I0 + W>(cf[1]) * v[W][1];
  });
#pragma unroll
  for (int k = 2; k < NS; k++) fma_bcast_steps<I0>(acc, cf[k], v[0][k], v[1][k], v[2][k], v[3][k]);
#pragma unroll
  for (int w = 0; w < 4; w++) acc[w] += first[w];
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
template <typename T, int NS, int LPC, bool FULL, bool VEC>
__global__ __launch_bounds__(64 * LPC) void k_ssm_fwd(SsmArgs a) {
  using P = Place<LPC>;
  constexpr int CW = P::CW, CH = P::CH, NT = P::NT, TL = SSM_TL, UPT = TL * CH / 4 / NT, YS = CH + 16;
  // tiles in flight: four, or two where a tile takes many registers
  constexpr int PF = NS == 4 && UPT * (int)sizeof(Raw4<T>) <= 16 ? 4 : 2;
  constexpr bool AHEAD = NS == 4;  // more states give independent work by themselves
  constexpr unsigned E = sizeof(T);
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
  unsigned ou[UPT], od[UPT], oz[UPT], oy[UPT];  // byte offsets in the tile's rows
  float ub[UPT][4], uD[UPT][4];
#pragma unroll
  for (int q = 0; q < UPT; q++) {
    const int id = q * NT + tid;
    ur[q] = id / (CH / 4);
    uc[q] = (id % (CH / 4)) * 4;
    unv[q] = w.nch - uc[q];
    const unsigned ch = (unsigned)(w.ch0 + uc[q]) * E;
    ou[q] = ur[q] * (unsigned)a.u.st * E + ch;
    od[q] = ur[q] * (unsigned)a.dt.st * E + ch;
    oz[q] = ur[q] * (unsigned)a.z.st * E + ch;
    oy[q] = ur[q] * (unsigned)a.y.st * E + ch;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const bool in = i < unv[q];
      ub[q][i] = in && a.bias ? a.bias[w.ch0 + uc[q] + i] : 0.f;
      uD[q][i] = FULL && in && a.Dk ? a.Dk[w.ch0 + uc[q] + i] : 0.f;
    }
  }
  const unsigned oB = ((lane & 15) * (unsigned)a.Bm.st + w.g * a.N + n0) * E;
  const unsigned oC = ((lane & 15) * (unsigned)a.Cm.st + w.g * a.N + n0) * E;
  const bool gate = a.z.p != nullptr;
  const int nt = (a.T + TL - 1) / TL;

  struct Slot {
    Raw4<T> u[UPT], d[UPT], z[UPT], B[NS / 4], C[NS / 4];
  };
  Slot ring[PF];
  auto load_tile = [&](Slot &s, int tile) PR_INLINE {
    const int t0 = w.t0 + tile * TL, left = end - t0;
    const SRsrc rd = rows_of<T>(a.dt, w.b, t0), ru = rows_of<T>(a.u, w.b, t0), rz = rows_of<T>(a.z, w.b, t0);
    const SRsrc rB = rows_of<T>(a.Bm, w.b, t0), rC = rows_of<T>(a.Cm, w.b, t0);
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const int nv = ur[q] < left ? unv[q] : 0;
      s.d[q] = load4<T, VEC>(rd, od[q], nv);
      s.u[q] = load4<T, VEC>(ru, ou[q], nv);
      if (FULL) s.z[q] = load4<T, VEC>(rz, oz[q], nv);
    }
#pragma unroll
    for (int q = 0; q < NS / 4; q++) {
      const int nv = (lane & 15) < left ? a.N - n0 - q * 4 : 0;
      s.B[q] = load4<T, VEC>(rB, oB + q * 4 * E, nv);
      if (FULL) s.C[q] = load4<T, VEC>(rC, oC + q * 4 * E, nv);
    }
  };
  Raw4<T> pu[UPT], pz[UPT];  // of the tile whose outputs are due
  auto output = [&](int tile) PR_INLINE {
    if constexpr (FULL) {
      const int t0 = w.t0 + tile * TL;
      const SRsrc ry = rows_of<T>(a.y, w.b, t0);
#pragma unroll
      for (int q = 0; q < UPT; q++) {
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          float v = fmaf(uD[q][i], pu[q].get(i), sy[tile & 1][ur[q]][uc[q] + i]);
          if (gate) {
            const float zz = pz[q].get(i);
            v *= zz * fsigm(zz);
          }
          o[i] = t0 + ur[q] < end ? v : 0.f;
        }
        store4<T, VEC>(ry, oy[q], o, t0 + ur[q] < w.t1 ? unv[q] : 0);
      }
    }
  };

  auto run_tile = [&](Slot &s, int tile, auto parity) PR_INLINE {
    constexpr int p = decltype(parity)::value;
    const int t0 = w.t0 + tile * TL;
    float B[NS], C[NS];
#pragma unroll
    for (int k = 0; k < NS; k++) {
      B[k] = s.B[k / 4].get(k % 4);
      if (FULL) C[k] = s.C[k / 4].get(k % 4);
    }
    Raw4<T> cu[UPT], cz[UPT];
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const bool live = t0 + ur[q] < end;
      float dx[8];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float v = s.d[q].get(i) + ub[q][i];
        if (a.softplus) v = softplus_f(v);
        v = live && i < unv[q] ? v : 0.f;
        dx[2 * i] = v;
        dx[2 * i + 1] = v * s.u[q].get(i);
      }
      float4 *o = reinterpret_cast<float4 *>(&sdx[p][ur[q]][uc[q]]);
      o[0] = make_float4(dx[0], dx[1], dx[2], dx[3]);
      o[1] = make_float4(dx[4], dx[5], dx[6], dx[7]);
      cu[q] = s.u[q];
      if (FULL) cz[q] = s.z[q];
    }
    load_tile(s, tile + PF);
    lds_barrier();
    if (tile > 0) output(tile - 1);
    if constexpr (FULL) {
      const SRsrc rs = s_rsrc(a.states + ((long long)w.b * nt + t0 / TL) * dn, a.states != nullptr);
#pragma unroll
      for (int q = 0; q < NS / 4; q++)
        store4<float, VEC>(rs, ((unsigned)d * a.N + n0 + q * 4) * 4u, h + q * 4, on ? a.N - n0 - q * 4 : 0);
    }
    // Four steps at a time: the decays and inputs of the next four are made
    // while these run, so that no instruction waits for the one before it.
    float ea[AHEAD ? 2 : 1][4][NS], xb[AHEAD ? 2 : 1][4][NS];
    auto prepare = [&](auto quad) PR_INLINE {
      constexpr int Q = decltype(quad)::value;
      unroll_up<4>([&](auto within) PR_INLINE {
        constexpr int W = decltype(within)::value, I = Q * 4 + W;
        const float2 dx = sdx[p][I][c];
#pragma unroll
        for (int k = 0; k < NS; k++) {
          ea[AHEAD ? Q & 1 : 0][W][k] = __builtin_amdgcn_exp2f(dx.x * A2[k]);
          xb[AHEAD ? Q & 1 : 0][W][k] = row_bcast<I>(B[k]) * dx.y;
        }
        if (!FULL) dsum += dx.x;
      });
    };
    if constexpr (AHEAD) prepare(std::integral_constant<int, 0>{});
    unroll_up<TL / 4>([&](auto quad) PR_INLINE {
      constexpr int Q = decltype(quad)::value;
      if constexpr (!AHEAD) prepare(quad);
      else if constexpr (Q + 1 < TL / 4) prepare(std::integral_constant<int, Q + 1>{});
      float(&hs)[4][NS] = xb[AHEAD ? Q & 1 : 0];
#pragma unroll
      for (int w4 = 0; w4 < 4; w4++)
#pragma unroll
        for (int k = 0; k < NS; k++) {
          hs[w4][k] = fmaf(ea[AHEAD ? Q & 1 : 0][w4][k], h[k], hs[w4][k]);
          h[k] = hs[w4][k];
        }
      if constexpr (FULL) {
        float acc[4];
        sum_bcast<Q * 4, NS>(acc, C, hs);
#pragma unroll
        for (int q = 0; q < 4; q += LPC) sy[p][Q * 4 + q + j][c] = group_sums<LPC>(acc + q);
      }
    });
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      pu[q] = cu[q];
      if (FULL) pz[q] = cz[q];
    }
  };

  unroll_up<PF>([&](auto i) PR_INLINE { load_tile(ring[decltype(i)::value], decltype(i)::value); });
  for (int tile = 0; tile < ntiles; tile += PF)
    unroll_up<PF>([&](auto i) PR_INLINE {
      constexpr int I = decltype(i)::value;
      if (tile + I < ntiles) run_tile(ring[I], tile + I, std::integral_constant<int, I & 1>{});
    });
  if constexpr (FULL) {
    if (ntiles > 0) {
      lds_barrier();
      output(ntiles - 1);
    }
    // steps past the sequence's length
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t = w.t0 + ntiles * TL; t < w.t1; t += TL) {
      const SRsrc ry = rows_of<T>(a.y, w.b, t);
#pragma unroll
      for (int q = 0; q < UPT; q++) store4<T, VEC>(ry, oy[q], zero, t + ur[q] < w.t1 ? unv[q] : 0);
    }
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
template <typename T, int NS, int LPC, bool VEC>
__global__ __launch_bounds__(64 * LPC) void k_ssm_adj_agg(SsmArgs a) {
  using P = Place<LPC>;
  constexpr int CW = P::CW, CH = P::CH, NT = P::NT, TL = SSM_TL, UPT = TL * CH / 4 / NT;
  constexpr int PF = NS == 4 && UPT * (int)sizeof(Raw4<T>) <= 16 ? 4 : 2;
  constexpr bool AHEAD = NS == 4;
  constexpr unsigned E = sizeof(T);
  __shared__ float2 sde[2][TL][CH];  // delta, e
  const P w(a);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int j = lane / CW, c = wave * CW + lane % CW, n0 = j * NS;
  const bool on = c < w.nch, gate = a.z.p != nullptr;
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
  int ur[UPT], uc[UPT], unv[UPT];
  unsigned od[UPT], oy[UPT], oz[UPT];
  float ub[UPT][4];
#pragma unroll
  for (int q = 0; q < UPT; q++) {
    const int id = q * NT + tid;
    ur[q] = id / (CH / 4);
    uc[q] = (id % (CH / 4)) * 4;
    unv[q] = w.nch - uc[q];
    const unsigned ch = (unsigned)(w.ch0 + uc[q]) * E;
    od[q] = ur[q] * (unsigned)a.dt.st * E + ch;
    oy[q] = ur[q] * (unsigned)a.dy.st * E + ch;
    oz[q] = ur[q] * (unsigned)a.z.st * E + ch;
#pragma unroll
    for (int i = 0; i < 4; i++) ub[q][i] = i < unv[q] && a.bias ? a.bias[w.ch0 + uc[q] + i] : 0.f;
  }
  const unsigned oC = ((lane & 15) * (unsigned)a.Cm.st + w.g * a.N + n0) * E;
  struct Slot {
    Raw4<T> d[UPT], y[UPT], z[UPT], C[NS / 4];
  };
  Slot ring[PF];
  // tiles run from the last to the first; one before the first reads nothing
  auto load_tile = [&](Slot &s, int tile) PR_INLINE {
    const int t0 = w.t0 + (tile < 0 ? 0 : tile) * TL, left = tile < 0 ? 0 : end - t0;
    const SRsrc rd = rows_of<T>(a.dt, w.b, t0), ry = rows_of<T>(a.dy, w.b, t0), rz = rows_of<T>(a.z, w.b, t0);
    const SRsrc rC = rows_of<T>(a.Cm, w.b, t0);
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const int nv = ur[q] < left ? unv[q] : 0;
      s.d[q] = load4<T, VEC>(rd, od[q], nv);
      s.y[q] = load4<T, VEC>(ry, oy[q], nv);
      s.z[q] = load4<T, VEC>(rz, oz[q], nv);
    }
#pragma unroll
    for (int q = 0; q < NS / 4; q++)
      s.C[q] = load4<T, VEC>(rC, oC + q * 4 * E, (lane & 15) < left ? a.N - n0 - q * 4 : 0);
  };
  float dsum = 0.f;
  auto run_tile = [&](Slot &s, int tile, auto parity) PR_INLINE {
    constexpr int p = decltype(parity)::value;
    const int t0 = w.t0 + tile * TL;
    float C[NS];
#pragma unroll
    for (int k = 0; k < NS; k++) C[k] = s.C[k / 4].get(k % 4);
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const bool in = t0 + ur[q] < end && i < unv[q];
        float v = s.d[q].get(i) + ub[q][i];
        if (a.softplus) v = softplus_f(v);
        float e = s.y[q].get(i);
        if (gate) {
          const float zz = s.z[q].get(i);
          e *= zz * fsigm(zz);
        }
        o[2 * i] = in ? v : 0.f;
        o[2 * i + 1] = in ? e : 0.f;
      }
      float4 *q4 = reinterpret_cast<float4 *>(&sde[p][ur[q]][uc[q]]);
      q4[0] = make_float4(o[0], o[1], o[2], o[3]);
      q4[1] = make_float4(o[4], o[5], o[6], o[7]);
    }
    load_tile(s, tile - PF);
    lds_barrier();
    float ea[AHEAD ? 2 : 1][4][NS], ce[AHEAD ? 2 : 1][4][NS];  // decay, C e of four steps
    auto prepare = [&](auto quad) PR_INLINE {
      constexpr int Q = decltype(quad)::value;
      unroll_up<4>([&](auto within) PR_INLINE {
        constexpr int W = decltype(within)::value, I = Q * 4 + W;
        const float2 de = sde[p][I][c];
#pragma unroll
        for (int k = 0; k < NS; k++) {
          ea[AHEAD ? Q & 1 : 0][W][k] = __builtin_amdgcn_exp2f(de.x * A2[k]);
          ce[AHEAD ? Q & 1 : 0][W][k] = row_bcast<I>(C[k]) * de.y;
        }
        dsum += de.x;
      });
    };
    if constexpr (AHEAD) prepare(std::integral_constant<int, TL / 4 - 1>{});
    unroll_up<TL / 4>([&](auto quad) PR_INLINE {
      constexpr int Q = TL / 4 - 1 - decltype(quad)::value;
      if constexpr (!AHEAD) prepare(std::integral_constant<int, Q>{});
      else if constexpr (Q > 0) prepare(std::integral_constant<int, Q - 1>{});
#pragma unroll
      for (int w4 = 3; w4 >= 0; w4--)
#pragma unroll
        for (int k = 0; k < NS; k++) r[k] = ea[AHEAD ? Q & 1 : 0][w4][k] * (ce[AHEAD ? Q & 1 : 0][w4][k] + r[k]);
    });
  };
  unroll_up<PF>([&](auto i) PR_INLINE { load_tile(ring[decltype(i)::value], ntiles - 1 - decltype(i)::value); });
  for (int tile = ntiles - 1; tile >= 0; tile -= PF)
    unroll_up<PF>([&](auto i) PR_INLINE {
      constexpr int I = decltype(i)::value;
      if (tile - I >= 0) run_tile(ring[I], tile - I, std::integral_constant<int, I & 1>{});
    });
  const long long at = (long long)w.b * a.S + w.s;
  store_state<NS>(a.agg + at * dn + (long long)d * a.N, n0, a.N, on, r);
  if (j == 0 && on) a.sumd[at * a.D + d] = dsum;
}

// The gradients of one segment, 4 states per lane and group of states (NG
// groups of 4 LPC states one after the other).  Per tile the states of its 16
// steps are made again from the saved one that enters it and stay in
// registers with their decays for the walk back.
template <typename T, int NG, int LPC, bool VEC>
__global__ __launch_bounds__(64 * LPC) void k_ssm_adj(SsmArgs a) {
  using P = Place<LPC>;
  constexpr int CW = P::CW, CH = P::CH, NT = P::NT, TL = SSM_TL, UPT = TL * CH / 4 / NT, YS = CH + 16;
  constexpr int GP = 4 * LPC, NP = NG * GP;  // states of a group, padded number of states
  constexpr int PF = 2;                      // tiles in flight
  constexpr unsigned E = sizeof(T);
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
  const bool on = c < w.nch, gate = a.z.p != nullptr;
  const int d = w.ch0 + c;
  const int end = w.t1 < w.len ? w.t1 : w.len;
  const int ntiles = end > w.t0 ? (end - w.t0 + TL - 1) / TL : 0;
  const int nt = (a.T + TL - 1) / TL;
  const long long dn = (long long)a.D * a.N;
  const long long at = (long long)w.b * a.S + w.s;
  const bool odd1 = lane & 1, odd2 = lane & 2, odd4 = lane & 4, odd8 = lane & 8;

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
  // byte offset of unit q in the rows of a tile of array v
  auto off = [&](const View &v, int q) PR_INLINE {
    return (ur[q] * (unsigned)v.st + (unsigned)(w.ch0 + uc[q])) * E;
  };
  struct Slot {
    Raw4<T> u[UPT], d[UPT], y[UPT], z[UPT], B[NG], C[NG];
    Raw4<float> h[NG];
  };
  Slot ring[PF];
  auto load_tile = [&](Slot &s, int tile) PR_INLINE {
    const int t0 = w.t0 + (tile < 0 ? 0 : tile) * TL, left = tile < 0 ? 0 : end - t0;
    const SRsrc ru = rows_of<T>(a.u, w.b, t0), rd = rows_of<T>(a.dt, w.b, t0), ry = rows_of<T>(a.dy, w.b, t0);
    const SRsrc rz = rows_of<T>(a.z, w.b, t0), rB = rows_of<T>(a.Bm, w.b, t0), rC = rows_of<T>(a.Cm, w.b, t0);
    const SRsrc rh = s_rsrc(a.states + ((long long)w.b * nt + t0 / TL) * dn);
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const int nv = ur[q] < left ? unv[q] : 0;
      s.u[q] = load4<T, VEC>(ru, off(a.u, q), nv);
      s.d[q] = load4<T, VEC>(rd, off(a.dt, q), nv);
      s.y[q] = load4<T, VEC>(ry, off(a.dy, q), nv);
      s.z[q] = load4<T, VEC>(rz, off(a.z, q), nv);
    }
#pragma unroll
    for (int g = 0; g < NG; g++) {
      const int n0 = g * GP + j * 4, nv = (lane & 15) < left ? a.N - n0 : 0;
      s.B[g] = load4<T, VEC>(rB, ((lane & 15) * (unsigned)a.Bm.st + w.g * a.N + n0) * E, nv);
      s.C[g] = load4<T, VEC>(rC, ((lane & 15) * (unsigned)a.Cm.st + w.g * a.N + n0) * E, nv);
      s.h[g] = load4<float, VEC>(rh, ((unsigned)d * a.N + n0) * 4u, on && left > 0 ? a.N - n0 : 0);
    }
  };
  // of the tile that `output` finishes: its buffer may be refilled meanwhile
  Raw4<T> pu[UPT], pd[UPT], py[UPT], pz[UPT];
  float pdl[UPT][4], pe[UPT][4];
  // gradients of a finished tile from its sums
  auto output = [&](int tile) PR_INLINE {
    const int t0 = w.t0 + tile * TL;
    const Buf &f = buf[(ntiles - 1 - tile) & 1];
    const SRsrc ru = rows_of<T>(a.du, w.b, t0), rd = rows_of<T>(a.ddt, w.b, t0), rz = rows_of<T>(a.dz, w.b, t0);
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const int t = t0 + ur[q];
      const bool live = t < end;
      float du[4], ddt[4], dz[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int cc = uc[q] + i;
        const float u = pu[q].get(i), v = pd[q].get(i) + ub[q][i];
        const float e = pe[q][i], gb = f.sum[1][ur[q]][cc];
        const bool in = live && i < unv[q];
        du[i] = in ? fmaf(pdl[q][i], gb, uD[q][i] * e) : 0.f;
        float dd = fmaf(u, gb, f.sum[2][ur[q]][cc]);
        if (a.softplus) dd *= fsigm(v);
        ddt[i] = in ? dd : 0.f;
        dz[i] = 0.f;
        if (gate) {
          const float zz = pz[q].get(i), s = fsigm(zz);
          const float y0 = fmaf(uD[q][i], u, f.sum[0][ur[q]][cc]);
          dz[i] = in ? py[q].get(i) * y0 * (s * fmaf(zz, 1.f - s, 1.f)) : 0.f;
        }
        accD[q][i] = fmaf(e, in ? u : 0.f, accD[q][i]);
        accb[q][i] += ddt[i];
      }
      const int nv = t < w.t1 ? unv[q] : 0;
      store4<T, VEC>(ru, off(a.du, q), du, nv);
      store4<T, VEC>(rd, off(a.ddt, q), ddt, nv);
      store4<T, VEC>(rz, off(a.dz, q), dz, nv);
    }
    // the waves' dB | dC of each step, to this channel block's partial
    const int in = w.cb - w.g * a.cbg, left = end - t0;
    const SRsrc rp = s_rsrc(a.part + ((((long long)in * a.B + w.b) * a.T + t0) * a.G + w.g) * (2 * NP));
#pragma unroll
    for (int i0 = 0; i0 < TL * 2 * NP; i0 += NT) {
      const int i = i0 + tid, row = i / (2 * NP), n = i % (2 * NP);
      float v = f.bc[0][row][n];
#pragma unroll
      for (int m = 1; m < LPC; m++) v += f.bc[m][row][n];
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rp,
                                            row < left ? (unsigned)(row * a.G * 2 * NP + n) * 4u : S_OOB, 0, 0);
    }
  };

  auto run_tile = [&](Slot &s, int tile, auto parity) PR_INLINE {
    const int t0 = w.t0 + tile * TL;
    Buf &f = buf[decltype(parity)::value];
    float B[NG][4], C[NG][4], hin[NG][4];
#pragma unroll
    for (int g = 0; g < NG; g++)
#pragma unroll
      for (int k = 0; k < 4; k++) {
        B[g][k] = s.B[g].get(k);
        C[g][k] = s.C[g].get(k);
        hin[g][k] = s.h[g].get(k);
      }
    Raw4<T> cu[UPT], cd[UPT], cy[UPT], cz[UPT];
    float cdl[UPT][4], ce[UPT][4];
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const bool live = t0 + ur[q] < end;
      float dx[8];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float v = s.d[q].get(i) + ub[q][i];
        if (a.softplus) v = softplus_f(v);
        float e = s.y[q].get(i);
        if (gate) {
          const float zz = s.z[q].get(i);
          e *= zz * fsigm(zz);
        }
        const bool in = live && i < unv[q];
        v = in ? v : 0.f;
        dx[2 * i] = v;
        dx[2 * i + 1] = v * s.u[q].get(i);
        cdl[q][i] = v;
        ce[q][i] = in ? e : 0.f;
      }
      float4 *o = reinterpret_cast<float4 *>(&f.dx[ur[q]][uc[q]]);
      o[0] = make_float4(dx[0], dx[1], dx[2], dx[3]);
      o[1] = make_float4(dx[4], dx[5], dx[6], dx[7]);
      *reinterpret_cast<float4 *>(&f.e[ur[q]][uc[q]]) = make_float4(ce[q][0], ce[q][1], ce[q][2], ce[q][3]);
      cu[q] = s.u[q];
      cd[q] = s.d[q];
      cy[q] = s.y[q];
      cz[q] = s.z[q];
    }
    load_tile(s, tile - PF);
    lds_barrier();
    if (tile + 1 < ntiles) output(tile + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int g = 0; g < NG; g++) {
      float hs[TL][4], as[TL][4];
      float A2[4];
#pragma unroll
      for (int k = 0; k < 4; k++) A2[k] = A[g][k] * 1.4426950408889634f;
      // the states again; all decays and inputs of four steps before their chain
      unroll_up<TL / 4>([&](auto quad) PR_INLINE {
        constexpr int Q = decltype(quad)::value;
        unroll_up<4>([&](auto within) PR_INLINE {
          constexpr int I = Q * 4 + decltype(within)::value;
          const float2 dx = f.dx[I][c];
#pragma unroll
          for (int k = 0; k < 4; k++) {
            as[I][k] = __builtin_amdgcn_exp2f(dx.x * A2[k]);
            hs[I][k] = row_bcast<I>(B[g][k]) * dx.y;
          }
        });
        unroll_up<4>([&](auto within) PR_INLINE {
          constexpr int I = Q * 4 + decltype(within)::value;
#pragma unroll
          for (int k = 0; k < 4; k++)
            hs[I][k] = fmaf(as[I][k], I > 0 ? hs[I > 0 ? I - 1 : 0][k] : hin[g][k], hs[I][k]);
        });
        // keeps the compiler from spreading the steps' temporaries over the whole tile
        __builtin_amdgcn_sched_barrier(0);
      });
      unroll_up<TL / 4>([&](auto quad) PR_INLINE {
        constexpr int Q = TL / 4 - 1 - decltype(quad)::value;
        float gg[4][4], q4[4][4], sum[3][4];
        float2 dx[4];
        float e[4];
#pragma unroll
        for (int m = 0; m < 4; m++) {
          dx[m] = f.dx[Q * 4 + m][c];
          e[m] = f.e[Q * 4 + m][c];
        }
        // the chain: g = r + C e, r = a g
        unroll_up<4>([&](auto within) PR_INLINE {
          constexpr int W = 3 - decltype(within)::value, I = Q * 4 + W;
#pragma unroll
          for (int k = 0; k < 4; k++) gg[W][k] = r[g][k];
          fma_bcast_states<I>(gg[W], C[g], e[W]);
#pragma unroll
          for (int k = 0; k < 4; k++) {
            r[g][k] = as[I][k] * gg[W][k];
            q4[W][k] = r[g][k] * (I > 0 ? hs[I > 0 ? I - 1 : 0][k] : hin[g][k]);
            dA[g][k] = fmaf(dx[W].x, q4[W][k], dA[g][k]);
          }
        });
        float(&h4)[4][4] = *reinterpret_cast<float(*)[4][4]>(&hs[Q * 4]);
        sum_bcast<Q * 4, 4>(sum[0], C[g], h4);
        sum_bcast<Q * 4, 4>(sum[1], B[g], gg);
#pragma unroll
        for (int m = 0; m < 4; m++) {
          float v = A[g][0] * q4[m][0];
#pragma unroll
          for (int k = 1; k < 4; k++) v = fmaf(A[g][k], q4[m][k], v);
          sum[2][m] = v;
        }
#pragma unroll
        for (int m = 0; m < 3; m++)
#pragma unroll
          for (int q = 0; q < 4; q += LPC) {
            float &o = f.sum[m][Q * 4 + q + j][c];  // the same lane adds each group's part
            const float v = group_sums<LPC>(sum[m] + q);
            o = g > 0 ? o + v : v;
          }
        // dB and dC of two steps, 16 values, over the 16 channels of each row:
        // every level sums pairs of lanes and packs two values into one
        // register, so that lane l of a row ends with value l in the order below
#pragma unroll
        for (int s2 = 0; s2 < 4; s2 += 2) {
          float p8[8], p4[4], p2[2];
#pragma unroll
          for (int m = 0; m < 8; m++) {  // m: step (1 bit), dB or dC (1 bit), pair of states (1 bit)
            const int st = s2 + (m >> 2), cc = (m >> 1) & 1, k = (m & 1) * 2;
            const float v0 = cc ? e[st] * h4[st][k] : dx[st].y * gg[st][k];
            const float v1 = cc ? e[st] * h4[st][k + 1] : dx[st].y * gg[st][k + 1];
            p8[m] = (odd8 ? v1 : v0) + dpp_f<0x128>(odd8 ? v0 : v1);  // lanes 8 apart: row_ror:8
          }
#pragma unroll
          for (int m = 0; m < 4; m++)  // lanes 4 apart, in rows of 8: row_half_mirror then quad_perm 3210
            p4[m] = (odd4 ? p8[2 * m + 1] : p8[2 * m]) +
                    dpp_f<0x1b>(dpp_f<0x141>(odd4 ? p8[2 * m] : p8[2 * m + 1]));
#pragma unroll
          for (int m = 0; m < 2; m++)  // lanes 2 apart: quad_perm 2301
            p2[m] = (odd2 ? p4[2 * m + 1] : p4[2 * m]) + dpp_f<0x4e>(odd2 ? p4[2 * m] : p4[2 * m + 1]);
          // lanes 1 apart: quad_perm 1032
          float v = (odd1 ? p2[1] : p2[0]) + dpp_f<0xb1>(odd1 ? p2[0] : p2[1]);
          if constexpr (LPC <= 2) v += __shfl_xor(v, 16, 64);  // rows that hold other channels of the same states
          if constexpr (LPC == 1) v += __shfl_xor(v, 32, 64);
          // lane l: step bit l & 1, dB or dC bit l & 2, state bits l & 4 (high), l & 8 (low)
          const int l = lane & 15;
          if (lane % CW < 16)
            f.bc[wave][Q * 4 + s2 + (l & 1)][((l >> 1) & 1) * NP + g * GP + j * 4 + ((l >> 2) & 1) * 2 + (l >> 3)] = v;
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    }
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      pu[q] = cu[q];
      pd[q] = cd[q];
      py[q] = cy[q];
      pz[q] = cz[q];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        pdl[q][i] = cdl[q][i];
        pe[q][i] = ce[q][i];
      }
    }
  };
  unroll_up<PF>([&](auto i) PR_INLINE { load_tile(ring[decltype(i)::value], ntiles - 1 - decltype(i)::value); });
  for (int tile = ntiles - 1; tile >= 0; tile -= PF)
    unroll_up<PF>([&](auto i) PR_INLINE {
      constexpr int I = decltype(i)::value;
      if (tile - I >= 0) run_tile(ring[I], tile - I, std::integral_constant<int, I & 1>{});
    });
  if (ntiles > 0) {
    lds_barrier();
    output(0);
  }
  // steps past the length: zero gradients
  const float zero[4] = {0.f, 0.f, 0.f, 0.f};
  for (int t = w.t0 + ntiles * TL; t < w.t1; t += TL) {
    const SRsrc ru = rows_of<T>(a.du, w.b, t), rd = rows_of<T>(a.ddt, w.b, t), rz = rows_of<T>(a.dz, w.b, t);
#pragma unroll
    for (int q = 0; q < UPT; q++) {
      const int nv = t + ur[q] < w.t1 ? unv[q] : 0;
      store4<T, VEC>(ru, off(a.du, q), zero, nv);
      store4<T, VEC>(rd, off(a.ddt, q), zero, nv);
      store4<T, VEC>(rz, off(a.dz, q), zero, nv);
    }
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
template <typename T, int NS, int LPC, bool VEC>
hipError_t ssm_launch_geom(const SsmArgs &a, int what, hipStream_t s) {
  const dim3 grid((unsigned)((long long)a.B * a.S * a.G * a.cbg));
  switch (what) {
    case SSM_FWD: k_ssm_fwd<T, NS, LPC, true, VEC><<<grid, 64 * LPC, 0, s>>>(a); break;
    case SSM_FWD_AGG: k_ssm_fwd<T, NS, LPC, false, VEC><<<grid, 64 * LPC, 0, s>>>(a); break;
    case SSM_ADJ: k_ssm_adj<T, NS / 4, LPC, VEC><<<grid, 64 * LPC, 0, s>>>(a); break;
    default: k_ssm_adj_agg<T, NS, LPC, VEC><<<grid, 64 * LPC, 0, s>>>(a); break;
  }
  return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t ssm_launch(const SsmArgs &a, int what, hipStream_t s) {
  const SsmGeom g = ssm_geom(a.N);
  if (g.ns == 4 && g.lpc == 1) return ssm_launch_geom<T, 4, 1, VEC>(a, what, s);
  if (g.ns == 4 && g.lpc == 2) return ssm_launch_geom<T, 4, 2, VEC>(a, what, s);
  if (g.ns == 4) return ssm_launch_geom<T, 4, 4, VEC>(a, what, s);
  if (g.ns == 8) return ssm_launch_geom<T, 8, 4, VEC>(a, what, s);
  return ssm_launch_geom<T, 16, 4, VEC>(a, what, s);
}

}  // namespace pr
