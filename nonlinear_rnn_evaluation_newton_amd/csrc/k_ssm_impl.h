// Selective state space scan and its adjoint, per channel d and state n:
//   h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t,  y_t = (C_t h_t + D u_t) silu(z_t)
//
// Layout.  A block holds 64 channels and walks time in tiles of 16 steps.  A
// wavefront holds 16 of them; lane = 16 j + c keeps NS states of channel c in
// registers, and WS wavefronts share the channels' states: state
// (ws 4 + j) NS + k.  B_t and C_t are the same for every channel of a group:
// lane i of each 16-lane row holds its states' B and C of step i of the tile,
// and a step's products take them by a row broadcast inside the instruction,
// so they cost neither shared memory nor an instruction.  delta and delta u
// are made once for each (step, channel) by the block's threads, UC channels
// each, and read back from shared memory; the sum over states runs in the lane,
// then over the four rows by register swaps, four steps at a time, and over
// the WS wavefronts where the output is made.
//
// Bound by vector arithmetic: per (step, channel, state) a product, an
// exponential (two issue slots), a product and two fused multiply-adds; what
// the states of a (step, channel) share is nearly as much again at 16 states.
// Measured (bf16, 2048 channels, 16 states; calls one after another): 8 x 4096
// steps 343 us, 3.1e12 (step, channel, state) a second, vector instructions
// being issued in 82% of the cycles; with unaligned arrays, element by element,
// 587 us; 32 states 509 us, 64 states 882 us.  The adjoint of 4 x 2048 steps 236
// us (85% of the cycles), with two preparing passes of 32 and 37 us; of more
// states 340 us for each 16.
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
constexpr unsigned S_OOB = 0x80000000u;  // outside every resource
__device__ inline SRsrc s_rsrc(const void *base, bool on = true) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, on ? 0x7fffffff : 0, 0x00020000);
}

// U adjacent elements as they are stored, in whole registers
template <typename T, int U>
struct Raw {
  static constexpr int W = U * (int)sizeof(T) <= 4 ? 1 : U * (int)sizeof(T) / 4;
  unsigned v[W];
  __device__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(v[i]);
    else return __uint_as_float((i & 1) ? (v[i / 2] & 0xffff0000u) : (v[i / 2] << 16));
  }
  __device__ void set(const float *f) {
#pragma unroll
    for (int i = 0; i < W; i++) {
      if constexpr (sizeof(T) == 4) v[i] = __float_as_uint(f[i]);
      else v[i] = (unsigned)f2bf(f[2 * i]) | (U > 1 ? (unsigned)f2bf(f[U > 1 ? 2 * i + 1 : 0]) << 16 : 0u);
    }
  }
};
typedef unsigned su32x2 __attribute__((ext_vector_type(2)));
typedef unsigned su32x4 __attribute__((ext_vector_type(4)));
template <int BYTES>
__device__ inline void buf_load(unsigned *v, SRsrc r, unsigned at, unsigned so) {
  if constexpr (BYTES == 2) v[0] = __builtin_amdgcn_raw_buffer_load_b16(r, at, so, 0);
  if constexpr (BYTES == 4) v[0] = __builtin_amdgcn_raw_buffer_load_b32(r, at, so, 0);
  if constexpr (BYTES == 8) {
    const su32x2 x = __builtin_amdgcn_raw_buffer_load_b64(r, at, so, 0);
    v[0] = x.x; v[1] = x.y;
  }
  if constexpr (BYTES == 16) {
    const su32x4 x = __builtin_amdgcn_raw_buffer_load_b128(r, at, so, 0);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  }
}
// A 16-byte store has its whole offset in the vector register: its data must not
// be overwritten by the very next instruction, which the compiler sees to only
// where the scalar offset is absent (with one, saved states came out wrong in
// the last lanes where the next instruction took the first data register).
template <int BYTES>
__device__ inline void buf_store(const unsigned *v, SRsrc r, unsigned at, unsigned so) {
  if constexpr (BYTES == 2) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)v[0], r, at, so, 0);
  if constexpr (BYTES == 4) __builtin_amdgcn_raw_buffer_store_b32(v[0], r, at, so, 0);
  if constexpr (BYTES == 8) __builtin_amdgcn_raw_buffer_store_b64(su32x2{v[0], v[1]}, r, at, so, 0);
  if constexpr (BYTES == 16) __builtin_amdgcn_raw_buffer_store_b128(su32x4{v[0], v[1], v[2], v[3]}, r, at + so, 0, 0);
}

// nv elements (at most U) from byte `off` of the lane plus byte `so` of the
// wavefront on, 0 past them.  VEC: one access, nv is at least U or not
// positive; else element by element.
template <typename T, int U, bool VEC>
__device__ inline Raw<T, U> load_u(SRsrc r, unsigned off, unsigned so, int nv) {
  Raw<T, U> o;
  constexpr int E = sizeof(T);
  if constexpr (VEC && U * E > 16) {
#pragma unroll
    for (int q = 0; q < U / 4; q++) buf_load<16>(o.v + 4 * q, r, nv > 0 ? off + 16 * q : S_OOB, so);
  } else if constexpr (VEC || U == 1) {
    buf_load<U * E>(o.v, r, nv > 0 ? off : S_OOB, so);
  } else {
#pragma unroll
    for (int i = 0; i < U; i++) {
      unsigned e;
      buf_load<E>(&e, r, i < nv ? off + E * i : S_OOB, so);
      if constexpr (E == 4) o.v[i] = e;
      else if (i & 1) o.v[i / 2] |= e << 16;
      else o.v[i / 2] = e;
    }
  }
  return o;
}
template <typename T, int U, bool VEC>
__device__ inline void store_u(SRsrc r, unsigned off, unsigned so, const float *f, int nv) {
  Raw<T, U> o;
  constexpr int E = sizeof(T);
  o.set(f);
  if constexpr (VEC && U * E > 16) {
#pragma unroll
    for (int q = 0; q < U / 4; q++) buf_store<16>(o.v + 4 * q, r, nv > 0 ? off + 16 * q : S_OOB, so);
  } else if constexpr (VEC || U == 1) {
    buf_store<U * E>(o.v, r, nv > 0 ? off : S_OOB, so);
  } else {
#pragma unroll
    for (int i = 0; i < U; i++) {
      const unsigned e = E == 4 ? o.v[E == 4 ? i : 0] : o.v[i / 2] >> (16 * (i & 1));
      buf_store<E>(&e, r, i < nv ? off + E * i : S_OOB, so);
    }
  }
}

// An array from the segment's first step of sequence b on, and the bytes of a
// tile: a tile's place is a scalar offset (the host keeps a segment's extent
// below 2^31 bytes).
template <typename T>
struct Rows {
  SRsrc r;
  unsigned tile;
  __device__ Rows(const View &v, int b, int t0)
      : r(s_rsrc((const T *)v.p + b * v.sb + t0 * v.st, v.p != nullptr)), tile(SSM_TL * (unsigned)v.st * sizeof(T)) {}
};

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
// acc[w] += v[w] times c of lane I0 + w; the wait at the end is for the register
// swaps that may use the sums next.
template <int I0>
__device__ inline void fma_bcast_steps(float *acc, float c, float v0, float v1, float v2, float v3) {
  asm("s_nop 1\n\t"
      "v_fmac_f32_dpp %0, %4, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %1, %4, %6 row_newbcast:%10 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %2, %4, %7 row_newbcast:%11 row_mask:0xf bank_mask:0xf\n\t"
      "v_fmac_f32_dpp %3, %4, %8 row_newbcast:%12 row_mask:0xf bank_mask:0xf\n\t"
      "s_nop 1"
      : "+&v"(acc[0]), "+&v"(acc[1]), "+&v"(acc[2]), "+&v"(acc[3])
      : "v"(c), "v"(v0), "v"(v1), "v"(v2), "v"(v3), "n"(I0), "n"(I0 + 1), "n"(I0 + 2), "n"(I0 + 3));
}

// o[w][k] = v[w] times c[k] of lane I0 + w, for two k
template <int I0>
__device__ inline void mul_bcast_steps(float (*o)[2], const float *c, const float *v) {
  asm("s_nop 1\n\t"
      "v_mul_f32_dpp %0, %8, %10 row_newbcast:%14 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %1, %9, %10 row_newbcast:%14 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %2, %8, %11 row_newbcast:%15 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %3, %9, %11 row_newbcast:%15 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %4, %8, %12 row_newbcast:%16 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %5, %9, %12 row_newbcast:%16 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %6, %8, %13 row_newbcast:%17 row_mask:0xf bank_mask:0xf\n\t"
      "v_mul_f32_dpp %7, %9, %13 row_newbcast:%17 row_mask:0xf bank_mask:0xf"
      : "=&v"(o[0][0]), "=&v"(o[0][1]), "=&v"(o[1][0]), "=&v"(o[1][1]), "=&v"(o[2][0]), "=&v"(o[2][1]), "=&v"(o[3][0]),
        "=&v"(o[3][1])
      : "v"(c[0]), "v"(c[1]), "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "n"(I0), "n"(I0 + 1), "n"(I0 + 2), "n"(I0 + 3));
}

// The first two levels of sums over the 16 lanes of a row, 16 values to 4
// registers: lanes 8 apart (the row's upper half takes the odd values), then 4
// apart (the odd quads take the odd registers).  An instruction writes only the
// quads of its bank mask, so two of them sum and pack two values.  The first
// waits for its sources as above.
__device__ inline void fold_rows(float *o, const float *v) {
  float t[8];
#define PR_F8(o_, a_, b_)                                                                  \
  "v_add_f32_dpp %" #o_ ", %" #a_ ", %" #a_ " row_ror:8 row_mask:0xf bank_mask:0x3\n\t"     \
  "v_add_f32_dpp %" #o_ ", %" #b_ ", %" #b_ " row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
#define PR_F4(o_, a_, b_)                                                                  \
  "v_add_f32_dpp %" #o_ ", %" #a_ ", %" #a_ " row_shl:4 row_mask:0xf bank_mask:0x5\n\t"     \
  "v_add_f32_dpp %" #o_ ", %" #b_ ", %" #b_ " row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
  asm("s_nop 1\n\t" PR_F8(4, 12, 13) PR_F8(5, 14, 15) PR_F8(6, 16, 17) PR_F8(7, 18, 19) PR_F8(8, 20, 21)
          PR_F8(9, 22, 23) PR_F8(10, 24, 25) PR_F8(11, 26, 27) PR_F4(0, 4, 5) PR_F4(1, 6, 7) PR_F4(2, 8, 9)
              PR_F4(3, 10, 11)
      : "=&v"(o[0]), "=&v"(o[1]), "=&v"(o[2]), "=&v"(o[3]), "=&v"(t[0]), "=&v"(t[1]), "=&v"(t[2]), "=&v"(t[3]),
        "=&v"(t[4]), "=&v"(t[5]), "=&v"(t[6]), "=&v"(t[7])
      : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]), "v"(v[6]), "v"(v[7]), "v"(v[8]), "v"(v[9]),
        "v"(v[10]), "v"(v[11]), "v"(v[12]), "v"(v[13]), "v"(v[14]), "v"(v[15]));
#undef PR_F8
#undef PR_F4
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
// Sums over the four rows for four steps at once: the lanes of row j end with
// the sum of v[j].
__device__ inline float group_sums(const float *v) {
  return pair_sums(half_sums(v[0], v[2]), half_sums(v[1], v[3]));
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

// The step size and the gate's factor, chosen without a branch: the four
// channels of a unit run side by side.
template <typename T>
__device__ inline float delta_of(float v, bool sp) {
  float s = sizeof(T) == 4 ? softplus_f(v) : softplus_short(v);
  asm volatile("" : "+v"(s));  // keeps it out of a branch on sp
  return sp ? s : v;
}
__device__ inline float gate_of(float z, bool gate) {
  float s = z * fsigm(z);
  asm volatile("" : "+v"(s));
  return gate ? s : 1.f;
}

// acc[w] = sum over k of v[w][k] times the value of cf[k] that lane I0 + w of
// each row holds
template <int I0, int NS>
__device__ inline void sum_bcast(float *acc, const float *cf, const float (*v)[NS]) {
  unroll_up<4>([&](auto within) PR_INLINE {
    constexpr int W = decltype(within)::value;
    acc[W] = row_bcast<I0 + W>(cf[0]) * v[W][0];
  });
#pragma unroll
  for (int k = 1; k < NS; k++) fma_bcast_steps<I0>(acc, cf[k], v[0][k], v[1][k], v[2][k], v[3][k]);
}

// What a block works on: a channel block of one group, a time segment, a
// sequence; and a thread's part of it.
template <typename T, int WS>
struct Place {
  static constexpr int CH = 64, NT = 256 * WS, TL = SSM_TL, UC = TL * CH / NT;  // UC: channels of a thread's unit
  static constexpr unsigned E = sizeof(T);
  int b, s, cb, g, ch0, nch, t0, t1, len;  // ch0: first channel; nch: channels of the block
  int end, ntiles;                         // steps past `end` leave the state as it is
  int lane, j, c, ws, d;                   // scan: row, channel in the block and in all, part of the states
  bool on;                                 // the lane's channel exists
  int ur, uc, unv;                         // staging: step of the tile, first channel, channels that exist
  __device__ Place(const SsmArgs &a) {
    const unsigned ncb = (unsigned)(a.G * a.cbg);
    const unsigned i = blockIdx.x;
    cb = (int)(i % ncb);
    const unsigned bs = i / ncb;
    s = (int)(bs % (unsigned)a.segs) + a.seg0;
    b = (int)(bs / (unsigned)a.segs);
    g = cb / a.cbg;
    const int in = (cb - g * a.cbg) * CH;
    ch0 = g * a.dpg + in;
    nch = a.dpg - in < CH ? a.dpg - in : CH;
    t0 = s * a.seglen;
    t1 = a.T - t0 < a.seglen ? a.T : t0 + a.seglen;
    len = seq_len(a.lengths, b, a.T);
    end = t1 < len ? t1 : len;
    ntiles = end > t0 ? (end - t0 + TL - 1) / TL : 0;
    const int tid = threadIdx.x, wave = tid >> 6;
    lane = tid & 63;
    j = lane >> 4;
    c = (wave / WS) * 16 + (lane & 15);
    ws = wave % WS;
    d = ch0 + c;
    on = c < nch;
    ur = tid / (CH / UC);
    uc = (tid % (CH / UC)) * UC;
    unv = nch - uc;
  }
  // byte offset of the thread's unit in the rows of a tile
  __device__ unsigned unit(const View &v) const { return (ur * (unsigned)v.st + (unsigned)(ch0 + uc)) * E; }
  // byte offset of state n0 of the lane's step in the rows of a tile of B or C
  __device__ unsigned coef(const View &v, int N, int n0) const {
    return ((lane & 15) * (unsigned)v.st + (unsigned)(g * N + n0)) * E;
  }
  // a per-channel parameter of the unit, 0 where there is none
  __device__ void param(const float *p, float *o) const {
#pragma unroll
    for (int i = 0; i < UC; i++) o[i] = p && i < unv ? p[ch0 + uc + i] : 0.f;
  }
};

template <int NS>
__device__ inline void load_state(const float *p, int n0, int N, bool on, float *h) {
#pragma unroll
  for (int i = 0; i < NS; i++) h[i] = on && n0 + i < N ? p[n0 + i] : 0.f;
}
template <int NS>
__device__ inline void store_state(float *p, int n0, int N, bool on, const float *h) {
#pragma unroll
  for (int i = 0; i < NS; i++)
    if (on && n0 + i < N) p[n0 + i] = h[i];
}

// out[channel] = the sum over the rows of a tile, which different threads hold,
// through the block's shared memory
template <typename P, int UC>
__device__ inline void sum_rows(const P &w, const float *v, float *sh, float *out) {
  __syncthreads();
#pragma unroll
  for (int i = 0; i < UC; i++) sh[w.ur * P::CH + w.uc + i] = v[i];
  __syncthreads();
  const int cc = threadIdx.x;
  if (cc < w.nch) {
    float s = 0.f;
#pragma unroll
    for (int row = 0; row < P::TL; row++) s += sh[row * P::CH + cc];
    out[w.ch0 + cc] = s;
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// FULL: outputs, from the state that enters the segment (a.agg where S > 1,
// else h0).  Not FULL: the end state of a piece of a segment from zero, and its
// sum of delta.
template <typename T, int NS, int WS, bool FULL, bool VEC>
__global__ __launch_bounds__(256 * WS) void k_ssm_fwd(SsmArgs a) {
  using P = Place<T, WS>;
  constexpr int CH = P::CH, TL = P::TL, UC = P::UC, YS = CH + 16;
  constexpr int PF = NS <= 4 ? 4 : 2;   // tiles in flight
  constexpr bool AHEAD = NS <= 4;       // more states give independent work by themselves
  __shared__ float2 sdx[2][TL][CH];     // delta, delta u
  __shared__ float sy[FULL ? 2 : 1][FULL ? WS : 1][FULL ? TL : 1][YS];
  const P w(a);
  const int n0 = (w.ws * 4 + w.j) * NS;
  const long long dn = (long long)a.D * a.N;
  const bool gate = a.z.p != nullptr, sp = a.softplus != 0;
  const int nt = (a.T + TL - 1) / TL;

  float A2[NS], h[NS];
  load_state<NS>(a.A + (long long)w.d * a.N, n0, a.N, w.on, A2);
#pragma unroll
  for (int k = 0; k < NS; k++) A2[k] *= 1.4426950408889634f;
  if constexpr (FULL) {
    const float *hp = a.carry   ? a.carry + w.b * dn
                      : a.S > 1 ? a.agg + ((long long)w.b * a.SA + w.s * a.R) * dn
                      : a.h0    ? a.h0 + w.b * dn
                                : nullptr;
    load_state<NS>(hp + (long long)w.d * a.N, n0, a.N, w.on && hp, h);
  } else {
#pragma unroll
    for (int k = 0; k < NS; k++) h[k] = 0.f;
  }
  float dsum[UC] = {}, ub[UC], uD[UC];  // dsum: not FULL, of the staged units
  w.param(a.bias, ub);
  w.param(FULL ? a.Dk : nullptr, uD);

  struct Slot {
    Raw<T, UC> u, d, z;
    Raw<T, NS> B, C;
  };
  Slot ring[PF];
  const unsigned ou = w.unit(a.u), od = w.unit(a.dt), oz = w.unit(a.z), oy = w.unit(a.y);
  const unsigned oB = w.coef(a.Bm, a.N, n0), oC = w.coef(a.Cm, a.N, n0);
  const Rows<T> ru(a.u, w.b, w.t0), rd(a.dt, w.b, w.t0), rz(a.z, w.b, w.t0), ry(a.y, w.b, w.t0);
  const Rows<T> rB(a.Bm, w.b, w.t0), rC(a.Cm, w.b, w.t0);
  const SRsrc rs = s_rsrc(a.states + ((long long)w.b * nt + w.t0 / TL) * dn, a.states != nullptr);
  auto load_tile = [&](Slot &s, int tile) PR_INLINE {
    const int left = w.end - w.t0 - tile * TL;
    const int nv = w.ur < left ? w.unv : 0, nn = (w.lane & 15) < left ? a.N - n0 : 0;
    s.d = load_u<T, UC, VEC>(rd.r, od, tile * rd.tile, nv);
    s.u = load_u<T, UC, VEC>(ru.r, ou, tile * ru.tile, nv);
    if (FULL) s.z = load_u<T, UC, VEC>(rz.r, oz, tile * rz.tile, nv);
    s.B = load_u<T, NS, VEC>(rB.r, oB, tile * rB.tile, nn);
    if (FULL) s.C = load_u<T, NS, VEC>(rC.r, oC, tile * rC.tile, nn);
  };
  Raw<T, UC> pu{}, pz{}, cu{}, cz{};  // of the tile whose outputs are due, of the staged tile
  Raw<T, NS> tB, tC;
  auto output = [&](int tile) PR_INLINE {
    if constexpr (FULL) {
      const int t0 = w.t0 + tile * TL;
      float o[UC];
#pragma unroll
      for (int i = 0; i < UC; i++) {
        float v = sy[tile & 1][0][w.ur][w.uc + i];
#pragma unroll
        for (int m = 1; m < WS; m++) v += sy[tile & 1][FULL ? m : 0][w.ur][w.uc + i];
        v = fmaf(uD[i], pu.get(i), v) * gate_of(pz.get(i), gate);
        o[i] = t0 + w.ur < w.end ? v : 0.f;
      }
      // (the scalar offset stays inside the resource also where nothing is stored)
      store_u<T, UC, VEC>(ry.r, oy, (tile < 0 ? 0u : (unsigned)tile) * ry.tile, o,
                          tile >= 0 && t0 + w.ur < w.t1 ? w.unv : 0);
    }
  };
  auto stage = [&](Slot &s, int tile, auto parity) PR_INLINE {
    constexpr int p = decltype(parity)::value;
    const bool live = w.t0 + tile * TL + w.ur < w.end;
    tB = s.B;
    if (FULL) tC = s.C;
    float dx[2 * UC];
#pragma unroll
    for (int i = 0; i < UC; i++) {
      const float v = delta_of<T>(s.d.get(i) + ub[i], sp);
      dx[2 * i] = live && i < w.unv ? v : 0.f;
      dx[2 * i + 1] = dx[2 * i] * s.u.get(i);
      if (!FULL) dsum[i] += dx[2 * i];
    }
#pragma unroll
    for (int i = 0; i < UC; i += 2)
      *reinterpret_cast<float4 *>(&sdx[p][w.ur][w.uc + i]) =
          make_float4(dx[2 * i], dx[2 * i + 1], dx[2 * i + 2], dx[2 * i + 3]);
    cu = s.u;
    if (FULL) cz = s.z;
    load_tile(s, tile + PF);
  };
  // The scan of one tile; meanwhile the outputs of the one before it and the
  // staging of the one after it (slot `next`), which give independent work.
  auto run_tile = [&](Slot &next, int tile, auto parity) PR_INLINE {
    constexpr int p = decltype(parity)::value;
    float B[NS], C[NS];
#pragma unroll
    for (int k = 0; k < NS; k++) {
      B[k] = tB.get(k);
      if (FULL) C[k] = tC.get(k);
    }
    lds_barrier();
    output(tile - 1);
    pu = cu;
    pz = cz;
    stage(next, tile + 1, std::integral_constant<int, p ^ 1>{});
    if constexpr (FULL)
      store_u<float, NS, VEC>(rs, ((unsigned)w.d * a.N + n0) * 4u, tile * (unsigned)dn * 4u, h,
                              w.on && a.states ? a.N - n0 : 0);
    // Four steps at a time: the decays and inputs of the next four are made
    // while these run, so that no instruction waits for the one before it.
    float ea[AHEAD ? 2 : 1][4][NS], xb[AHEAD ? 2 : 1][4][NS];
    auto prepare = [&](auto quad) PR_INLINE {
      constexpr int Q = decltype(quad)::value;
      unroll_up<4>([&](auto within) PR_INLINE {
        constexpr int W = decltype(within)::value, I = Q * 4 + W;
        const float2 dx = sdx[p][I][w.c];
#pragma unroll
        for (int k = 0; k < NS; k++) {
          ea[AHEAD ? Q & 1 : 0][W][k] = __builtin_amdgcn_exp2f(dx.x * A2[k]);
          xb[AHEAD ? Q & 1 : 0][W][k] = row_bcast<I>(B[k]) * dx.y;
        }
      });
    };
    if constexpr (AHEAD) prepare(std::integral_constant<int, 0>{});
    unroll_up<TL / 4>([&](auto quad) PR_INLINE {
      constexpr int Q = decltype(quad)::value;
      if constexpr (!AHEAD) prepare(quad);
      else if constexpr (Q + 1 < TL / 4) prepare(std::integral_constant<int, Q + 1>{});
      float(&hs)[4][NS] = xb[AHEAD ? Q & 1 : 0];
#pragma unroll
      for (int m = 0; m < 4; m++)
#pragma unroll
        for (int k = 0; k < NS; k++) {
          hs[m][k] = fmaf(ea[AHEAD ? Q & 1 : 0][m][k], h[k], hs[m][k]);
          h[k] = hs[m][k];
        }
      if constexpr (FULL) {
        float acc[4];
        sum_bcast<Q * 4, NS>(acc, C, hs);
        sy[p][w.ws][Q * 4 + w.j][w.c] = group_sums(acc);
      }
    });
  };

  unroll_up<PF>([&](auto i) PR_INLINE { load_tile(ring[decltype(i)::value], decltype(i)::value); });
  stage(ring[0], 0, std::integral_constant<int, 0>{});
  for (int tile = 0; tile < w.ntiles; tile += PF)
    unroll_up<PF>([&](auto i) PR_INLINE {
      constexpr int I = decltype(i)::value;
      if (tile + I < w.ntiles) run_tile(ring[(I + 1) % PF], tile + I, std::integral_constant<int, I & 1>{});
    });
  if constexpr (FULL) {
    if (w.ntiles > 0) {
      lds_barrier();
      output(w.ntiles - 1);
    }
    // steps past the sequence's length
    const float zero[UC] = {};
    for (int tile = w.ntiles; w.t0 + tile * TL < w.t1; tile++)
      store_u<T, UC, VEC>(ry.r, oy, tile * ry.tile, zero, w.t0 + tile * TL + w.ur < w.t1 ? w.unv : 0);
    const int last = w.len > 0 ? (w.len - 1) / a.seglen : 0;
    if (a.hlast && w.s == last)
      store_state<NS>(a.hlast + w.b * dn + (long long)w.d * a.N, n0, a.N, w.on, h);
    if (a.carry) store_state<NS>(a.carry + w.b * dn + (long long)w.d * a.N, n0, a.N, w.on, h);
  } else {
    const long long at = (long long)w.b * a.SA + w.s;
    store_state<NS>(a.agg + at * dn + (long long)w.d * a.N, n0, a.N, w.on, h);
    sum_rows<P, UC>(w, dsum, &sdx[0][0][0].x, a.sumd + at * a.D);
  }
}

// ---------------------------------------------------------------------------
// adjoint
// ---------------------------------------------------------------------------
// With e_t = dy_t silu(z_t), the adjoint state g_t = C_t e_t + a_{t+1} g_{t+1}
// runs backwards; r_t = a_t g_t is what a step hands to the one before it.
// This pass: a piece's r at its first step from zero behind it.
template <typename T, int NS, int WS, bool VEC>
__global__ __launch_bounds__(256 * WS) void k_ssm_adj_agg(SsmArgs a) {
  using P = Place<T, WS>;
  constexpr int CH = P::CH, TL = P::TL, UC = P::UC;
  constexpr int PF = NS <= 4 ? 4 : 2;
  constexpr bool AHEAD = NS <= 4;
  __shared__ float2 sde[2][TL][CH];  // delta, e
  const P w(a);
  const int n0 = (w.ws * 4 + w.j) * NS;
  const long long dn = (long long)a.D * a.N;
  const bool gate = a.z.p != nullptr, sp = a.softplus != 0;
  float A2[NS], r[NS], ub[UC], dsum[UC] = {};
  load_state<NS>(a.A + (long long)w.d * a.N, n0, a.N, w.on, A2);
  w.param(a.bias, ub);
#pragma unroll
  for (int k = 0; k < NS; k++) {
    A2[k] *= 1.4426950408889634f;
    r[k] = 0.f;
  }
  struct Slot {
    Raw<T, UC> d, y, z;
    Raw<T, NS> C;
  };
  Slot ring[PF];
  Raw<T, NS> tC;
  const unsigned od = w.unit(a.dt), oy = w.unit(a.dy), oz = w.unit(a.z), oC = w.coef(a.Cm, a.N, n0);
  const Rows<T> rd(a.dt, w.b, w.t0), ry(a.dy, w.b, w.t0), rz(a.z, w.b, w.t0), rC(a.Cm, w.b, w.t0);
  // tiles run from the last to the first; one before the first reads nothing
  auto load_tile = [&](Slot &s, int tile) PR_INLINE {
    const int left = tile < 0 ? 0 : w.end - w.t0 - tile * TL;
    const int nv = w.ur < left ? w.unv : 0;
    const unsigned at = tile < 0 ? 0u : (unsigned)tile;
    s.d = load_u<T, UC, VEC>(rd.r, od, at * rd.tile, nv);
    s.y = load_u<T, UC, VEC>(ry.r, oy, at * ry.tile, nv);
    s.z = load_u<T, UC, VEC>(rz.r, oz, at * rz.tile, nv);
    s.C = load_u<T, NS, VEC>(rC.r, oC, at * rC.tile, (w.lane & 15) < left ? a.N - n0 : 0);
  };
  auto stage = [&](Slot &s, int tile, auto parity) PR_INLINE {
    constexpr int p = decltype(parity)::value;
    const bool live = tile >= 0 && w.t0 + tile * TL + w.ur < w.end;
    tC = s.C;
    float o[2 * UC];
#pragma unroll
    for (int i = 0; i < UC; i++) {
      const bool in = live && i < w.unv;
      const float v = delta_of<T>(s.d.get(i) + ub[i], sp), e = s.y.get(i) * gate_of(s.z.get(i), gate);
      o[2 * i] = in ? v : 0.f;
      dsum[i] += o[2 * i];
      o[2 * i + 1] = in ? e : 0.f;
    }
#pragma unroll
    for (int i = 0; i < UC; i += 2)
      *reinterpret_cast<float4 *>(&sde[p][w.ur][w.uc + i]) =
          make_float4(o[2 * i], o[2 * i + 1], o[2 * i + 2], o[2 * i + 3]);
    load_tile(s, tile - PF);
  };
  auto run_tile = [&](Slot &next, int tile, auto parity) PR_INLINE {
    constexpr int p = decltype(parity)::value;
    float C[NS];
#pragma unroll
    for (int k = 0; k < NS; k++) C[k] = tC.get(k);
    lds_barrier();
    stage(next, tile - 1, std::integral_constant<int, p ^ 1>{});
    float ea[AHEAD ? 2 : 1][4][NS], ce[AHEAD ? 2 : 1][4][NS];  // decay, C e of four steps
    auto prepare = [&](auto quad) PR_INLINE {
      constexpr int Q = decltype(quad)::value;
      unroll_up<4>([&](auto within) PR_INLINE {
        constexpr int W = decltype(within)::value, I = Q * 4 + W;
        const float2 de = sde[p][I][w.c];
#pragma unroll
        for (int k = 0; k < NS; k++) {
          ea[AHEAD ? Q & 1 : 0][W][k] = __builtin_amdgcn_exp2f(de.x * A2[k]);
          ce[AHEAD ? Q & 1 : 0][W][k] = row_bcast<I>(C[k]) * de.y;
        }
      });
    };
    if constexpr (AHEAD) prepare(std::integral_constant<int, TL / 4 - 1>{});
    unroll_up<TL / 4>([&](auto quad) PR_INLINE {
      constexpr int Q = TL / 4 - 1 - decltype(quad)::value;
      if constexpr (!AHEAD) prepare(std::integral_constant<int, Q>{});
      else if constexpr (Q > 0) prepare(std::integral_constant<int, Q - 1>{});
#pragma unroll
      for (int m = 3; m >= 0; m--)
#pragma unroll
        for (int k = 0; k < NS; k++) r[k] = ea[AHEAD ? Q & 1 : 0][m][k] * (ce[AHEAD ? Q & 1 : 0][m][k] + r[k]);
    });
  };
  const int n = w.ntiles;
  unroll_up<PF>([&](auto i) PR_INLINE { load_tile(ring[decltype(i)::value], n - 1 - decltype(i)::value); });
  stage(ring[0], n - 1, std::integral_constant<int, 0>{});
  for (int tile = n - 1; tile >= 0; tile -= PF)
    unroll_up<PF>([&](auto i) PR_INLINE {
      constexpr int I = decltype(i)::value;
      if (tile - I >= 0) run_tile(ring[(I + 1) % PF], tile - I, std::integral_constant<int, I & 1>{});
    });
  const long long at = (long long)w.b * a.SA + w.s;
  store_state<NS>(a.agg + at * dn + (long long)w.d * a.N, n0, a.N, w.on, r);
  sum_rows<P, UC>(w, dsum, &sde[0][0][0].x, a.sumd + at * a.D);
}

// The gradients of one segment.  A wavefront keeps two states per lane, 8 WS
// states in all, from state a.n_off on.  Per tile the states of its 16 steps
// are made again from the saved one that enters it and stay in registers with
// their decays for the walk back.  MULTI: more than 16 states, one launch for
// each 16; the sums over states go through a.acc from one to the next, and the
// last one makes the outputs.  (One kernel for all of more than 16 states did
// not fit the registers, and its copies of registers to make room were made
// where a branch on lanes joined, with lanes still off: there are no such
// branches in the loops of these kernels.)
template <typename T, int WS, bool MULTI, bool VEC>
__global__ __launch_bounds__(256 * WS) void k_ssm_adj(SsmArgs a) {
  using P = Place<T, WS>;
  constexpr int CH = P::CH, TL = P::TL, UC = P::UC, NT = P::NT, YS = CH + 16, NS = 2;
  constexpr int GP = 4 * WS * NS;                // states of a launch
  constexpr int RS = WS == 1 && !VEC ? 1 : 2;    // tiles in flight, as the registers allow
  constexpr unsigned E = sizeof(T);
  struct Buf {
    float2 dx[TL][CH];                      // delta, delta u
    float e[TL][CH];
    float sum[3][WS][TL][YS];               // sums over a wavefront's states: C h, B g, A r h_{t-1}
    float bc[4][TL][2 * GP];                // dB | dC of 16 channels
  };
  __shared__ Buf buf[2];
  const P w(a);
  const bool gate = a.z.p != nullptr, sp = a.softplus != 0;
  const int nt = (a.T + TL - 1) / TL, nl = (w.ws * 4 + w.j) * NS;  // nl: the lane's first state of these
  const long long dn = (long long)a.D * a.N;
  const long long at = a.carry ? w.b : (long long)w.b * a.S + w.s;
  const bool odd1 = w.lane & 1, odd2 = w.lane & 2;

  const int n0 = a.n_off + nl, NPT = a.NPT;

  float A[NS], A2[NS], r[NS], dA[NS];
  load_state<NS>(a.A + (long long)w.d * a.N, n0, a.N, w.on, A);
  const float *rp0 = a.carry    ? a.carry + w.b * dn
                     : a.S > 1  ? a.agg + ((long long)w.b * a.SA + (w.s + 1) * a.R - 1) * dn
                     : a.dhlast ? a.dhlast + w.b * dn
                                : nullptr;
  load_state<NS>(rp0 + (long long)w.d * a.N, n0, a.N, w.on && rp0, r);
#pragma unroll
  for (int k = 0; k < NS; k++) {
    dA[k] = 0.f;
    A2[k] = A[k] * 1.4426950408889634f;
  }
  float ub[UC], uD[UC], accD[UC] = {}, accb[UC] = {};
  w.param(a.bias, ub);
  w.param(a.Dk, uD);

  struct Slot {
    Raw<T, UC> u, d, y, z;
  };
  struct Coef {  // of one tile
    Raw<T, NS> B, C;
    Raw<float, NS> h;
  };
  Slot ring[RS];
  Coef coef[2];
  const unsigned ou = w.unit(a.u), od = w.unit(a.dt), oy = w.unit(a.dy), oz = w.unit(a.z);
  const unsigned oB = w.coef(a.Bm, a.N, n0), oC = w.coef(a.Cm, a.N, n0), oh = ((unsigned)w.d * a.N + n0) * 4u;
  const unsigned odu = w.unit(a.du), odd = w.unit(a.ddt), odz = w.unit(a.dz);
  const Rows<T> ru(a.u, w.b, w.t0), rd(a.dt, w.b, w.t0), ry(a.dy, w.b, w.t0), rz(a.z, w.b, w.t0);
  const Rows<T> rB(a.Bm, w.b, w.t0), rC(a.Cm, w.b, w.t0);
  const Rows<T> rdu(a.du, w.b, w.t0), rdd(a.ddt, w.b, w.t0), rdz(a.dz, w.b, w.t0);
  const SRsrc rh = s_rsrc(a.states + ((long long)w.b * nt + w.t0 / TL) * dn);
  const SRsrc rp = s_rsrc(a.part + ((((long long)(w.cb - w.g * a.cbg) * a.B + w.b) * a.T + w.t0) * a.G + w.g) * (2 * NPT) + a.n_off);
  // tiles run from the last to the first; one before the first reads nothing
  auto load_tile = [&](Slot &s, int tile) PR_INLINE {
    const int left = tile < 0 ? 0 : w.end - w.t0 - tile * TL;
    const int nv = w.ur < left ? w.unv : 0;
    const unsigned at = tile < 0 ? 0u : (unsigned)tile;
    s.u = load_u<T, UC, VEC>(ru.r, ou, at * ru.tile, nv);
    s.d = load_u<T, UC, VEC>(rd.r, od, at * rd.tile, nv);
    s.y = load_u<T, UC, VEC>(ry.r, oy, at * ry.tile, nv);
    s.z = load_u<T, UC, VEC>(rz.r, oz, at * rz.tile, nv);
  };
  auto load_coef = [&](Coef &s, int tile) PR_INLINE {
    const int left = tile < 0 ? 0 : w.end - w.t0 - tile * TL;
    const unsigned at = tile < 0 ? 0u : (unsigned)tile;
    const int nn = a.N - n0, on = (w.lane & 15) < left ? nn : 0;
    s.B = load_u<T, NS, VEC>(rB.r, oB, at * rB.tile, on);
    s.C = load_u<T, NS, VEC>(rC.r, oC, at * rC.tile, on);
    s.h = load_u<float, NS, VEC>(rh, oh, at * (unsigned)dn * 4u, w.on && left > 0 ? nn : 0);
  };
  // c: of the staged tile, p: of the tile whose outputs are due (its buffer may
  // be refilled meanwhile)
  Raw<T, UC> cu{}, cd{}, cy{}, cz{}, pu{}, pd{}, py{}, pz{};
  float cdl[UC] = {}, ce[UC] = {}, pdl[UC] = {}, pe[UC] = {};
  auto stage = [&](Slot &s, int tile, auto parity) PR_INLINE {
    Buf &f = buf[decltype(parity)::value];
    const bool live = tile >= 0 && w.t0 + tile * TL + w.ur < w.end;
#pragma unroll
    for (int i = 0; i < UC; i++) {
      const bool in = live && i < w.unv;
      const float v = delta_of<T>(s.d.get(i) + ub[i], sp), e = s.y.get(i) * gate_of(s.z.get(i), gate);
      cdl[i] = in ? v : 0.f;
      ce[i] = in ? e : 0.f;
    }
#pragma unroll
    for (int i = 0; i < UC; i += 2) {
      *reinterpret_cast<float4 *>(&f.dx[w.ur][w.uc + i]) =
          make_float4(cdl[i], cdl[i] * s.u.get(i), cdl[i + 1], cdl[i + 1] * s.u.get(i + 1));
      *reinterpret_cast<float2 *>(&f.e[w.ur][w.uc + i]) = make_float2(ce[i], ce[i + 1]);
    }
    cu = s.u;
    cd = s.d;
    cy = s.y;
    cz = s.z;
    load_tile(s, tile - RS);
  };
  // a.acc: [B][T][3][D]
  const SRsrc racc = s_rsrc(MULTI ? a.acc + ((long long)w.b * a.T + w.t0) * 3 * a.D : nullptr, MULTI);
  const unsigned oacc = ((unsigned)w.ur * 3 * a.D + w.ch0 + w.uc) * 4u, tacc = TL * 3u * a.D * 4u;
  // gradients of a finished tile from its sums (parity of its buffer)
  auto output = [&](int tile, int parity) PR_INLINE {
    const bool any = tile < w.ntiles;
    const int t0 = w.t0 + tile * TL, t = t0 + w.ur, left = any ? w.end - t0 : 0;
    const Buf &f = buf[parity];
    float du[UC], ddt[UC], dz[UC], sums[3][UC];
#pragma unroll
    for (int m = 0; m < 3; m++) {
#pragma unroll
      for (int i = 0; i < UC; i++) {
        sums[m][i] = f.sum[m][0][w.ur][w.uc + i];
#pragma unroll
        for (int q = 1; q < WS; q++) sums[m][i] += f.sum[m][q][w.ur][w.uc + i];
      }
      if constexpr (MULTI) {
        const int nv = w.ur < left ? w.unv : 0;
        const Raw<float, UC> x = load_u<float, UC, VEC>(racc, oacc + m * a.D * 4u, tile * tacc, a.n_off > 0 ? nv : 0);
#pragma unroll
        for (int i = 0; i < UC; i++) sums[m][i] += x.get(i);
        store_u<float, UC, VEC>(racc, oacc + m * a.D * 4u, tile * tacc, sums[m], a.last ? 0 : nv);
      }
    }
    const bool fin = !MULTI || a.last != 0;
#pragma unroll
    for (int i = 0; i < UC; i++) {
      const bool in = w.ur < left && i < w.unv && fin;
      const float sum[3] = {sums[0][i], sums[1][i], sums[2][i]};
      const float u = pu.get(i), v = pd.get(i) + ub[i], e = pe[i], zz = pz.get(i);
      const float sg = fsigm(v), s = fsigm(zz), y0 = fmaf(uD[i], u, sum[0]);
      float o[3] = {fmaf(pdl[i], sum[1], uD[i] * e), fmaf(u, sum[1], sum[2]) * (sp ? sg : 1.f),
                    py.get(i) * y0 * (s * fmaf(zz, 1.f - s, 1.f))};  // dz: stored where there is a gate
      // (values of their own, so that they are selected below and not branched to)
      asm volatile("" : "+v"(o[0]), "+v"(o[1]), "+v"(o[2]));
      du[i] = in ? o[0] : 0.f;
      ddt[i] = in ? o[1] : 0.f;
      dz[i] = in ? o[2] : 0.f;
      accD[i] = fmaf(e, in ? u : 0.f, accD[i]);
      accb[i] += ddt[i];
    }
    const int nv = any && t < w.t1 && fin ? w.unv : 0;
    store_u<T, UC, VEC>(rdu.r, odu, tile * rdu.tile, du, nv);
    store_u<T, UC, VEC>(rdd.r, odd, tile * rdd.tile, ddt, nv);
    store_u<T, UC, VEC>(rdz.r, odz, tile * rdz.tile, dz, nv);
    // dB | dC of each step, to this channel block's partial
#pragma unroll
    for (int i0 = 0; i0 < TL * 2 * GP; i0 += NT) {
      const int i = i0 + (int)threadIdx.x, row = i / (2 * GP), n = i % (2 * GP);
      const float v = (f.bc[0][row][n] + f.bc[1][row][n]) + (f.bc[2][row][n] + f.bc[3][row][n]);
      const unsigned uv = __float_as_uint(v);
      buf_store<4>(&uv, rp, row < left ? (unsigned)(row * a.G * 2 * NPT + (n < GP ? n : NPT + n - GP)) * 4u : S_OOB,
                   tile * (unsigned)(TL * a.G * 2 * NPT) * 4u);
    }
  };

  auto run_tile = [&](Slot &next, int tile, auto parity) PR_INLINE {
    constexpr int p = decltype(parity)::value;
    Buf &f = buf[p];
    lds_barrier();
    output(tile + 1, p ^ 1);
    pu = cu;
    pd = cd;
    py = cy;
    pz = cz;
#pragma unroll
    for (int i = 0; i < UC; i++) {
      pdl[i] = cdl[i];
      pe[i] = ce[i];
    }
    stage(next, tile - 1, std::integral_constant<int, p ^ 1>{});
    {
      float hs[TL][NS], as[TL][NS], B[NS], C[NS], hin[NS];
      Coef &cf = coef[p];
#pragma unroll
      for (int k = 0; k < NS; k++) {
        B[k] = cf.B.get(k);
        C[k] = cf.C.get(k);
        hin[k] = cf.h.get(k);
      }
      load_coef(cf, tile - 2);
      // the states again; the decays and inputs of four steps before their chain
      unroll_up<TL / 4>([&](auto quad) PR_INLINE {
        constexpr int Q = decltype(quad)::value;
        float x[4];
#pragma unroll
        for (int m = 0; m < 4; m++) {
          const float2 dx = f.dx[Q * 4 + m][w.c];
          x[m] = dx.y;
#pragma unroll
          for (int k = 0; k < NS; k++) as[Q * 4 + m][k] = __builtin_amdgcn_exp2f(dx.x * A2[k]);
        }
        mul_bcast_steps<Q * 4>(&hs[Q * 4], B, x);
        unroll_up<4>([&](auto within) PR_INLINE {
          constexpr int I = Q * 4 + decltype(within)::value;
#pragma unroll
          for (int k = 0; k < NS; k++)
            hs[I][k] = fmaf(as[I][k], I > 0 ? hs[I > 0 ? I - 1 : 0][k] : hin[k], hs[I][k]);
        });
        // keeps the steps' temporaries from spreading over the whole tile
        __builtin_amdgcn_sched_barrier(0);
      });
      // (a value of its own: sharing the broadcasts of the first pass would keep
      // them in registers, as instructions apart)
#pragma unroll
      for (int k = 0; k < NS; k++) asm volatile("" : "+v"(B[k]));
      unroll_up<TL / 4>([&](auto quad) PR_INLINE {
        constexpr int Q = TL / 4 - 1 - decltype(quad)::value;
        float gg[4][NS], q4[4][NS], sum[3][4];
        float2 dx[4];
        float e[4];
#pragma unroll
        for (int m = 0; m < 4; m++) {
          dx[m] = f.dx[Q * 4 + m][w.c];
          e[m] = f.e[Q * 4 + m][w.c];
        }
        // the chain: g = r + C e, r = a g
        unroll_up<4>([&](auto within) PR_INLINE {
          constexpr int W = 3 - decltype(within)::value, I = Q * 4 + W;
#pragma unroll
          for (int k = 0; k < NS; k++) {
            gg[W][k] = fmaf(row_bcast<I>(C[k]), e[W], r[k]);
            r[k] = as[I][k] * gg[W][k];
            q4[W][k] = r[k] * (I > 0 ? hs[I > 0 ? I - 1 : 0][k] : hin[k]);
            dA[k] = fmaf(dx[W].x, q4[W][k], dA[k]);
          }
        });
        float(&h4)[4][NS] = *reinterpret_cast<float(*)[4][NS]>(&hs[Q * 4]);
        sum_bcast<Q * 4, NS>(sum[0], C, h4);
        sum_bcast<Q * 4, NS>(sum[1], B, gg);
#pragma unroll
        for (int m = 0; m < 4; m++) {
          float v = A[0] * q4[m][0];
#pragma unroll
          for (int k = 1; k < NS; k++) v = fmaf(A[k], q4[m][k], v);
          sum[2][m] = v;
        }
#pragma unroll
        for (int m = 0; m < 3; m++) f.sum[m][w.ws][Q * 4 + w.j][w.c] = group_sums(sum[m]);
        // dB and dC of four steps, 16 values, over the 16 channels of each row:
        // every level sums pairs of lanes and packs two values into one
        // register, so that each lane of a row ends with the sum of one value
        float v16[16], p4[4], p2[2];
#pragma unroll
        for (int m = 0; m < 8; m++) {  // m: step (2 bits), dB or dC (1 bit)
          const int st = m >> 1;
          v16[2 * m] = (m & 1) ? e[st] * h4[st][0] : dx[st].y * gg[st][0];
          v16[2 * m + 1] = (m & 1) ? e[st] * h4[st][1] : dx[st].y * gg[st][1];
        }
        fold_rows(p4, v16);
#pragma unroll
        for (int m = 0; m < 2; m++)  // lanes 2 apart: quad_perm 2301
          p2[m] = (odd2 ? p4[2 * m + 1] : p4[2 * m]) + dpp_f<0x4e>(odd2 ? p4[2 * m] : p4[2 * m + 1]);
        // lanes 1 apart: quad_perm 1032
        const float v = (odd1 ? p2[1] : p2[0]) + dpp_f<0xb1>(odd1 ? p2[0] : p2[1]);
        // lane l of a row: step bits l & 1 (high), l & 2 (low), dB or dC l & 4, state l & 8
        const int l = w.lane & 15;
        f.bc[w.c >> 4][Q * 4 + (l & 1) * 2 + ((l >> 1) & 1)][((l >> 2) & 1) * GP + nl + (l >> 3)] = v;
        __builtin_amdgcn_sched_barrier(0);
      });
    }
  };
  const int n = w.ntiles;
  unroll_up<RS>([&](auto i) PR_INLINE { load_tile(ring[decltype(i)::value], n - 1 - decltype(i)::value); });
  load_coef(coef[0], n - 1);
  load_coef(coef[1], n - 2);
  stage(ring[0], n - 1, std::integral_constant<int, 0>{});
  for (int tile = n - 1; tile >= 0; tile -= 2)
    unroll_up<2>([&](auto i) PR_INLINE {
      constexpr int I = decltype(i)::value;
      if (tile - I >= 0) run_tile(ring[(I + 1) % RS], tile - I, std::integral_constant<int, I>{});
    });
  if (n > 0) {
    lds_barrier();
    output(0, (n - 1) & 1);
  }
  // steps past the length: zero gradients
  const float zero[UC] = {};
  for (int tile = n; w.t0 + tile * TL < w.t1; tile++) {
    const int nv = w.t0 + tile * TL + w.ur < w.t1 && (!MULTI || a.last) ? w.unv : 0;
    store_u<T, UC, VEC>(rdu.r, odu, tile * rdu.tile, zero, nv);
    store_u<T, UC, VEC>(rdd.r, odd, tile * rdd.tile, zero, nv);
    store_u<T, UC, VEC>(rdz.r, odz, tile * rdz.tile, zero, nv);
  }
  if (a.accum) {
    float before[NS];
    load_state<NS>(a.pA + at * dn + (long long)w.d * a.N, n0, a.N, w.on, before);
#pragma unroll
    for (int k = 0; k < NS; k++) dA[k] += before[k];
  }
  store_state<NS>(a.pA + at * dn + (long long)w.d * a.N, n0, a.N, w.on, dA);
  if (a.dh0 && w.s == 0) store_state<NS>(a.dh0 + w.b * dn + (long long)w.d * a.N, n0, a.N, w.on, r);
  if (a.carry) store_state<NS>(a.carry + w.b * dn + (long long)w.d * a.N, n0, a.N, w.on, r);
  if (MULTI && !a.last) return;
  // dD and the bias' gradient: over the tile's rows, which different threads hold
  __syncthreads();
  float *red = reinterpret_cast<float *>(&buf[0]);  // [2][TL][CH]
#pragma unroll
  for (int i = 0; i < UC; i++) {
    red[w.ur * CH + w.uc + i] = accD[i];
    red[(TL + w.ur) * CH + w.uc + i] = accb[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * CH; i += NT) {
    const int m = i / CH, cc = i % CH;
    if (cc < w.nch) {
      float v = 0.f;
#pragma unroll
      for (int row = 0; row < TL; row++) v += red[(m * TL + row) * CH + cc];
      float *o = a.pD + (at * 2 + m) * a.D + w.ch0 + cc;
      *o = a.accum ? *o + v : v;
    }
  }
}

// ---------------------------------------------------------------------------
template <typename T, int NS, int WS, bool VEC>
hipError_t ssm_go(SsmArgs a, int what, hipStream_t s) {
  // no segment starts from the last one's end state (the first one's, backwards)
  const bool part = what == SSM_FWD_AGG || what == SSM_ADJ_AGG;
  a.segs = part ? a.SA - a.R : a.S;
  a.seg0 = what == SSM_ADJ_AGG ? a.R : a.win;
  if (part) a.seglen /= a.R;
  const dim3 grid((unsigned)((long long)a.B * a.segs * a.G * a.cbg));
  constexpr bool MULTI = NS > 2;
  switch (what) {
    case SSM_FWD: k_ssm_fwd<T, NS, WS, true, VEC><<<grid, 256 * WS, 0, s>>>(a); break;
    case SSM_FWD_AGG: k_ssm_fwd<T, NS, WS, false, VEC><<<grid, 256 * WS, 0, s>>>(a); break;
    case SSM_ADJ:
      a.NPT = 4 * NS * WS;
      for (a.n_off = 0; a.n_off < a.N; a.n_off += 8 * WS) {
        a.last = a.n_off + 8 * WS >= a.N;
        k_ssm_adj<T, WS, MULTI, VEC><<<grid, 256 * WS, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
      }
      return hipSuccess;
    default: k_ssm_adj_agg<T, NS, WS, VEC><<<grid, 256 * WS, 0, s>>>(a); break;
  }
  return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t ssm_launch(const SsmArgs &a, int what, hipStream_t s) {
  const SsmGeom g = ssm_geom(a.N);
  if (g.ns == 2 && g.ws == 1) return ssm_go<T, 2, 1, VEC>(a, what, s);
  if (g.ns == 2) return ssm_go<T, 2, 2, VEC>(a, what, s);
  if (g.ns == 4) return ssm_go<T, 4, 2, VEC>(a, what, s);
  return ssm_go<T, 8, 2, VEC>(a, what, s);
}

}  // namespace pr
