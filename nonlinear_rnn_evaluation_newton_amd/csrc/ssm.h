// Selective state space scan: arguments shared by its kernels and the ABI
// layer (k_ssm.hip), and the device helpers that several of them use.
#pragma once

#include "internal.h"

namespace pr {

// A [B, T, channels] array: element (b, t, c) at p[b * sb + t * st + c].
struct View {
  void *p;
  long long sb, st;
};

constexpr int SSM_TL = 16;  // steps per tile, and between two saved states

struct SsmArgs {
  View u, dt, z, Bm, Cm, y;          // z.p may be null
  View dy, du, ddt, dz, dB, dC;      // adjoint; outputs may be null
  const float *A, *Dk, *bias, *h0;   // Dk, bias, h0 may be null
  const int *lengths;                // may be null
  float *hlast, *states;             // may be null (states is required by the adjoint)
  const float *dhlast;               // adjoint, may be null
  float *dh0;                        // adjoint, may be null
  float *agg, *sumd;                 // time split: per (b, piece) end, then entering, states [D][N]; sums of delta [D]
  float *part;                       // adjoint: dB | dC partials [block of the group][B][T][G][2 NP]
  float *pA, *pD;                    // adjoint: [B S][D][N] and [B S][2][D] partials of dA, dD | dbias
  int B, T, D, N, G, softplus;
  int dpg, cbg;                      // channels per group, channel blocks per group
  int S, seglen;                     // time segments and their steps (a multiple of SSM_TL)
  int R, SA;                         // pieces of a segment in the passes that prepare the split, S R
  float *acc;                        // adjoint of more than 16 states: sums over states, [B][T][3][D]
  int n_off, last, NPT;              // its launches: first state, whether the last, padded number of states
  int segs, seg0;                    // segments or pieces of a launch and the first of them (set by the launcher)
  // long time strides: the segments are launched one after another (S = 1)
  float *carry;                      // null, or [B][D][N]: the state that enters the segment, then the one that leaves it
  int win, accum;                    // the segment; adjoint: whether dA, dD and dbias go on from what pA and pD hold
  int vec;                           // all arrays may be moved in vectors of four
};

// States per lane and wavefronts per channel of the scan kernels for N states
// (four lanes of a wavefront share a channel).  Sixteen states on one wavefront
// of four each would take fewer instructions, but leave one wavefront a SIMD:
// 366 against 342 us also where the blocks fill the device (8 x 4096 x 2048), and
// the adjoint has registers for two states a lane only.
struct SsmGeom {
  int ns, ws;
};
inline SsmGeom ssm_geom(int N) {
  if (N <= 8) return {2, 1};
  if (N <= 16) return {2, 2};
  if (N <= 32) return {4, 2};
  return {8, 2};
}

enum { SSM_FWD = 0, SSM_FWD_AGG = 1, SSM_ADJ = 2, SSM_ADJ_AGG = 3 };
// _vec: a.vec, every array may be moved in vectors of four
hipError_t launch_ssm_bf16(const SsmArgs &a, int what, hipStream_t s);
hipError_t launch_ssm_bf16_vec(const SsmArgs &a, int what, hipStream_t s);
hipError_t launch_ssm_f32(const SsmArgs &a, int what, hipStream_t s);
hipError_t launch_ssm_f32_vec(const SsmArgs &a, int what, hipStream_t s);

// out[j] = sum over p of part[p * stride + j], j < cols, added in order in 64 bits
hipError_t launch_part_sum(const float *part, int P, long long stride, long long cols, float *out, hipStream_t s);

// e^x with a relative error near 1e-7 for any |x| below 80: the product with
// log2(e) is carried in two words, which a single rounding of a large
// argument would lose.
__device__ inline float exp_acc(float x) {
  const float L = 1.44269502162933349609f, Ll = 1.92596299112661746887e-8f;
  const float p = x * L;
  float r = fmaf(x, L, -p);
  r = fmaf(x, Ll, r);
  const float e = __builtin_amdgcn_exp2f(p);
  // an infinite argument gives r = NaN, where e is already the answer
  return fabsf(x) < 128.f ? fmaf(e, r * 0.6931471805599453f, e) : e;
}

// log(1 + e) for 0 <= e <= 1: the logarithm of the rounded sum u, and what its
// rounding left out, e - (u - 1), over u.  That quotient is taken without the
// division: where u is not near 1 the term is below 2^-24 of the result.
__device__ inline float log1p_unit(float e) {
  const float u = 1.f + e;
  return fmaf(__builtin_amdgcn_logf(u), 0.6931471805599453f, e - (u - 1.f));
}

__device__ inline float softplus_f(float v) {
  const float l = log1p_unit(exp_acc(-fabsf(v)));
  return (v > 0.f ? v : 0.f) + l;  // a NaN comes through l
}

// The same with a plain product for the exponential's argument: its error of
// |v| 2^-24 is far below that of a v that was stored in 8 significant bits,
// and five instructions fewer.
__device__ inline float softplus_short(float v) {
  const float l = log1p_unit(fexp(-fabsf(v)));
  return (v > 0.f ? v : 0.f) + l;
}

// Steps of sequence b: all T, or its length, held to 0..T.
__device__ inline int seq_len(const int *lengths, int b, int T) {
  const int n = lengths ? lengths[b] : T;
  return n < 0 ? 0 : n > T ? T : n;
}

}  // namespace pr
