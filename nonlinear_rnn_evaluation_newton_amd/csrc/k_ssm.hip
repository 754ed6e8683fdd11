// Selective state space scan: the C entry points, the kernels that join the
// time segments and add the partial sums, and the single-token step.
#include <string>

#include "pararnn.h"
#include "ssm.h"
#include "vec.h"

namespace pr {

// ---------------------------------------------------------------------------
// joining the pieces
// ---------------------------------------------------------------------------
// agg[b][s] (end state of piece s from zero) becomes the state that enters
// piece s; a piece's factor is exp(A sum of delta).  REV: the same from the
// last piece back, for the adjoint's carry.  One thread per (b, d, n).
// The factor is applied as its root, twice: over a whole piece it may pass the
// range of fp32, for states that grow (A > 0), where the state that it meets is
// small enough for the step by step product to stay inside.  The root is held
// to finite values, so that a state of 0 stays 0, as it does step by step, and
// any other overflows (a NaN of the sum comes through the end state).
template <bool REV>
__global__ void k_ssm_join(const float *__restrict__ A, const float *__restrict__ first,
                           const float *__restrict__ sumd, float *__restrict__ agg, int B, int D, int N, int S) {
  const long long dn = (long long)D * N, i = flat_block() * 256 + threadIdx.x;
  if (i >= B * dn) return;
  const long long b = i / dn, e = i % dn;
  const int d = (int)(e / N);
  const float Ah = A[e] * (0.5f * 1.4426950408889634f);
  float carry = first ? first[i] : 0.f;
  const float *sd = sumd + b * S * D + d;
  float *ag = agg + b * S * dn + e;
  constexpr int U = 8;  // pieces whose loads are in flight together
  for (int s0 = 0; s0 < S; s0 += U) {
    float v[U], m[U];
#pragma unroll
    for (int q = 0; q < U; q++) {
      const int s = REV ? S - 1 - s0 - q : s0 + q;
      const bool in = s0 + q < S;
      // (the last one in this order has no sum: nothing follows it)
      v[q] = in && s0 + q + 1 < S ? ag[s * dn] : 0.f;
      m[q] = in && s0 + q + 1 < S ? sd[(long long)s * D] : 0.f;
    }
#pragma unroll
    for (int q = 0; q < U; q++) {
      const int s = REV ? S - 1 - s0 - q : s0 + q;
      if (s0 + q < S) {
        ag[s * dn] = carry;
        const float f = fminf(__builtin_amdgcn_exp2f(m[q] * Ah), 3.402823466e38f);
        carry = fmaf(f, f * carry, v[q]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// the adjoint's last sums, one launch
// ---------------------------------------------------------------------------
struct SsmSums {
  const float *part, *pA, *pD;  // as in SsmArgs
  const int *lengths;
  View dB, dC;
  float *dA, *dD, *dbias;       // may be null
  int nblk, B, T, G, N, NP, P, D;
  unsigned bc_blocks, a_blocks;  // blocks of the first two kinds, of which the first walk their outputs
};

// out[j] = the sum over p of part[p * stride + j], in 64 bits in a fixed order:
// COLS columns by SL slices of the partials per block, eight loads in flight
template <int COLS, int SL>
__device__ inline void part_sum(const float *__restrict__ part, int P, long long stride, long long cols, long long blk,
                                float *__restrict__ out) {
  __shared__ double sh[SL][COLS];
  const int x = threadIdx.x % COLS, y = threadIdx.x / COLS;
  const long long j = blk * COLS + x;
  double s = 0;
  if (j < cols)
    for (int p0 = y; p0 < P; p0 += 8 * SL) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; q++) v[q] = p0 + SL * q < P ? part[(p0 + SL * q) * stride + j] : 0.f;
#pragma unroll
      for (int q = 0; q < 8; q++) s += (double)v[q];
    }
  sh[y][x] = s;
  for (int h = SL / 2; h >= 1; h >>= 1) {
    __syncthreads();
    if (y < h) sh[y][x] += sh[y + h][x];
  }
  if (y == 0 && j < cols) out[j] = (float)sh[0][x];
}

// Blocks of three kinds: dB and dC of each (b, t, group, n) over the group's
// channel blocks; dA over the (b, segment) partials; dD, then dbias, likewise.
template <typename T>
__global__ __launch_bounds__(256) void k_ssm_sums(SsmSums a) {
  if (blockIdx.x >= a.bc_blocks) {
    const unsigned i = blockIdx.x - a.bc_blocks;
    if (i < a.a_blocks) {
      part_sum<32, 8>(a.pA, a.P, (long long)a.D * a.N, (long long)a.D * a.N, i, a.dA);
    } else {
      const unsigned m = (i - a.a_blocks) & 1, blk = (i - a.a_blocks) >> 1;
      float *o = m ? a.dbias : a.dD;
      if (o) part_sum<32, 8>(a.pD + (long long)m * a.D, a.P, 2LL * a.D, a.D, blk, o);
    }
    return;
  }
  const long long rows = (long long)a.B * a.T * a.G, cols = 2LL * a.NP;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < rows * cols; i += a.bc_blocks * 256LL) {
    const int n2 = (int)(i % cols), n = n2 % a.NP;
    if (n >= a.N) continue;
    const long long row = i / cols, bt = row / a.G;
    const int g = (int)(row % a.G), t = (int)(bt % a.T), b = (int)(bt / a.T);
    const View &v = n2 < a.NP ? a.dB : a.dC;
    if (!v.p) continue;
    float s = 0.f;
    if (t < seq_len(a.lengths, b, a.T)) {
#pragma unroll 8
      for (int k = 0; k < a.nblk; k++) s += a.part[k * rows * cols + i];
    }
    stf((T *)v.p, b * v.sb + t * v.st + (long long)g * a.N + n, s);
  }
}

// for many partials of few columns
__global__ __launch_bounds__(1024) void k_part_sum(const float *part, int P, long long stride, long long cols, float *out) {
  part_sum<16, 64>(part, P, stride, cols, flat_block(), out);
}

hipError_t launch_part_sum(const float *part, int P, long long stride, long long cols, float *out, hipStream_t s) {
  if (cols < 1) return hipSuccess;
  k_part_sum<<<flat_grid((cols + 15) / 16), 1024, 0, s>>>(part, P, stride, cols, out);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// one token
// ---------------------------------------------------------------------------
struct SsmStepArgs {
  const void *u, *dt, *z, *Bm, *Cm;
  void *y;
  long long su, sdt, sz, sB, sC, sy;  // row strides
  const float *A, *Dk, *bias;
  float *state;
  const int *slots;
  int B, D, N, G, nslots, softplus;
};

// LG lanes (a power of two) per channel, 4 states each; the state is read and
// written once, 16 bytes a lane where N is a multiple of 4.
template <typename T, int LG>
__global__ __launch_bounds__(256) void k_ssm_step(SsmStepArgs a) {
  const int lane = threadIdx.x % LG;
  const int d = (int)(blockIdx.x * (256 / LG) + threadIdx.x / LG), b = blockIdx.y;
  const bool on = d < a.D;
  const int slot = a.slots ? a.slots[b] : b;
  const bool live = slot >= 0 && slot < a.nslots;
  const int dd = on ? d : 0;
  float acc = 0.f, u = 0.f, zz = 0.f;
  if (live && on) {
    u = ldf((const T *)a.u, b * a.su + dd);
    float v = ldf((const T *)a.dt, b * a.sdt + dd) + (a.bias ? a.bias[dd] : 0.f);
    if (a.z) zz = ldf((const T *)a.z, b * a.sz + dd);
    if (a.softplus) v = softplus_f(v);
    const float x = v * u;
    const int g = dd / (a.D / a.G), n0 = lane * 4;
    const T *bp = (const T *)a.Bm + b * a.sB + (long long)g * a.N;
    const T *cp = (const T *)a.Cm + b * a.sC + (long long)g * a.N;
    const float *ap = a.A + (long long)dd * a.N;
    float *hp = a.state + ((long long)slot * a.D + dd) * a.N;
    float h[4], A[4];
    const bool v4 = (a.N & 3) == 0 && n0 < a.N;
    if (v4) {
      const float4 h4 = *reinterpret_cast<const float4 *>(hp + n0), a4 = *reinterpret_cast<const float4 *>(ap + n0);
      h[0] = h4.x; h[1] = h4.y; h[2] = h4.z; h[3] = h4.w;
      A[0] = a4.x; A[1] = a4.y; A[2] = a4.z; A[3] = a4.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; k++) {
        h[k] = n0 + k < a.N ? hp[n0 + k] : 0.f;
        A[k] = n0 + k < a.N ? ap[n0 + k] : 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float bb = n0 + k < a.N ? ldf(bp, n0 + k) : 0.f, cc = n0 + k < a.N ? ldf(cp, n0 + k) : 0.f;
      h[k] = fmaf(__builtin_amdgcn_exp2f(v * (A[k] * 1.4426950408889634f)), h[k], x * bb);
      acc = fmaf(cc, h[k], acc);
    }
    if (v4) {
      *reinterpret_cast<float4 *>(hp + n0) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; k++)
        if (n0 + k < a.N) hp[n0 + k] = h[k];
    }
  }
#pragma unroll
  for (int o = LG / 2; o >= 1; o >>= 1) acc += __shfl_xor(acc, o, 64);
  if (lane == 0 && on) {
    float y = 0.f;
    if (live) {
      y = a.Dk ? fmaf(a.Dk[d], u, acc) : acc;
      if (a.z) y *= zz * fsigm(zz);
    }
    stf((T *)a.y, b * a.sy + d, y);
  }
}

template <typename T>
hipError_t launch_step(const SsmStepArgs &a, hipStream_t s) {
  const int q = (a.N + 3) / 4;
#define PR_STEP(LG)                                                                           \
  {                                                                                           \
    k_ssm_step<T, LG><<<dim3((unsigned)((a.D + 256 / LG - 1) / (256 / LG)), (unsigned)a.B), 256, 0, s>>>(a); \
    return hipGetLastError();                                                                 \
  }
  if (q <= 1) PR_STEP(1)
  if (q <= 2) PR_STEP(2)
  if (q <= 4) PR_STEP(4)
  if (q <= 8) PR_STEP(8)
  PR_STEP(16)
#undef PR_STEP
}

}  // namespace pr

using namespace pr;

namespace {

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

#define HIPCHK(expr)                                                                        \
  do {                                                                                      \
    hipError_t e_ = (expr);                                                                 \
    if (e_ != hipSuccess) return fail(PR_EHIP, "%s: %s", #expr, hipGetErrorString(e_));     \
  } while (0)

struct SsmPlan {
  int cbg = 0, NP = 0, S = 1, seglen = 0, R = 1;
  size_t off_agg = 0, off_sumd = 0, off_part = 0, off_pA = 0, off_pD = 0, off_acc = 0, fwd_bytes = 0, adj_bytes = 0;
};

// Time segments for `blocks` blocks over T steps: a block for each CU, at
// least four tiles each; a segment's extent in any array below 2^31 bytes (16
// steps are).
// (1 x 32768 x 256 in fp32: 90 us with 64 segments, 289 with 16, 2613 with one;
// training on 4 x 2048 x 2048, 128 blocks: 411 us with two, 643 with one.)
// Between 129 and 255 blocks two segments take as many rounds of the device as
// one of twice the length, and their preparation is lost: 8 x 2048 steps of 1536
// channels, 192 blocks, 203 us, 171 unsplit; training 750 and 652.  Below, 5 of
// those sequences, 120 blocks: with three segments 146 and 522 us, with two 123
// and 411, with one 171 and 644.
// Two segments leave half of the CUs idle in the pass that prepares the split,
// which one segment of the two takes part in: it takes that one in two pieces
// (training on 4 x 2048 x 2048: 411 us, 470 in one piece).
void split_time(long long blocks, int T, long long max_tile_bytes, int *S, int *seglen, int *R) {
  const long long tiles = (T + SSM_TL - 1) / SSM_TL;
  long long s = (256 + blocks - 1) / blocks;
  const long long most = (tiles + 3) / 4;
  if (s > most) s = most;
  if (s < 1) s = 1;
  long long per = (tiles + s - 1) / s;
  const long long fit = ((1LL << 31) - (1LL << 30)) / max_tile_bytes;
  if (per > fit) per = fit;
  *R = s == 2 && per > 3 ? 2 : 1;
  if (*R == 2 && per < fit) per += per & 1;
  if (per & 1) *R = 1;
  *seglen = (int)(per * SSM_TL);
  *S = (int)((tiles + per - 1) / per);
}

// step: single tokens, T is not used and may be 0
int ssm_check(const pr_ssm_problem *p, bool step) {
  if (!p) return fail(PR_EINVAL, "problem is NULL");
  if (p->dtype != PR_F32 && p->dtype != PR_BF16) return fail(PR_EINVAL, "unknown dtype %d", p->dtype);
  if (p->B < 1 || p->T < (step ? 0 : 1) || p->D < 1 || p->N < 1 || p->G < 1)
    return fail(PR_EINVAL, "sizes must be >= 1 (B=%d T=%d D=%d N=%d G=%d)", p->B, p->T, p->D, p->N, p->G);
  if (p->D % p->G != 0) return fail(PR_EINVAL, "G = %d does not divide D = %d", p->G, p->D);
  if (p->N > 64) return fail(PR_EUNSUPPORTED, "N = %d states: at most 64", p->N);
  if (p->T > (1 << 30)) return fail(PR_EUNSUPPORTED, "T = %d: at most 2^30", p->T);
  if (p->D > (1 << 22)) return fail(PR_EUNSUPPORTED, "D = %d: at most 2^22", p->D);
  return PR_OK;
}

int ssm_plan(const pr_ssm_problem *p, SsmPlan *pl) {
  const int rc = ssm_check(p, false);
  if (rc != PR_OK) return rc;
  const SsmGeom g = ssm_geom(p->N);
  const int dpg = p->D / p->G;
  pl->cbg = (dpg + 63) / 64;
  pl->NP = 4 * g.ns * g.ws;
  const long long blocks = (long long)p->B * p->G * pl->cbg;
  const int esz = p->dtype == PR_BF16 ? 2 : 4;
  // rows as slices of projections up to four times as wide as they need be
  const long long width = p->D > (long long)p->G * p->N ? p->D : (long long)p->G * p->N;
  long long tile = SSM_TL * 4 * width * esz;
  if (tile < (long long)p->D * p->N * 4) tile = (long long)p->D * p->N * 4;
  if (tile < SSM_TL * 8LL * p->G * pl->NP) tile = SSM_TL * 8LL * p->G * pl->NP;
  if (p->N > 16 && tile < SSM_TL * 12LL * p->D) tile = SSM_TL * 12LL * p->D;
  if (tile > (1LL << 27)) return fail(PR_EUNSUPPORTED, "problem too large: %lld bytes in 16 steps", tile);
  split_time(blocks, p->T, tile, &pl->S, &pl->seglen, &pl->R);
  // a launch has 2^32 threads at most, 512 a block
  if (blocks * pl->S * pl->R >= (1LL << 23))
    return fail(PR_EUNSUPPORTED, "problem too large: %lld blocks of channels, %d segments", blocks, pl->S * pl->R);
  const size_t dn = (size_t)p->D * p->N, sm = pl->S > 1 ? pl->S * pl->R : 1;
  if ((double)p->B * sm * dn * 4 > 1e13 || (double)p->B * p->T * p->G * pl->cbg * pl->NP * 8 > 1e13)
    return fail(PR_EUNSUPPORTED, "problem too large");
  size_t o = 0;
  pl->off_agg = o; o = align256(o + p->B * sm * dn * 4);  // (one state: what goes from window to window)
  pl->off_sumd = o; o = align256(o + (sm > 1 ? p->B * sm * p->D * 4 : 0));
  pl->fwd_bytes = o > 256 ? o : 256;
  pl->off_part = o; o = align256(o + (size_t)pl->cbg * p->B * p->T * p->G * 2 * pl->NP * 4);
  pl->off_pA = o; o = align256(o + p->B * (size_t)pl->S * dn * 4);
  pl->off_pD = o; o = align256(o + p->B * (size_t)pl->S * 2 * p->D * 4);
  pl->off_acc = o; o = align256(o + (p->N > 16 ? (size_t)p->B * p->T * 3 * p->D * 4 : 0));
  pl->adj_bytes = o;
  return PR_OK;
}

View view(const pr_view *v, int T) {
  View r{nullptr, 0, 0};
  if (v && v->p) r = View{v->p, v->sb, T > 1 ? v->st : 0};  // an absent array has no strides, one step none over time
  return r;
}

// vectors of four elements may be used on it
bool vec4_ok(const View &v, int esz) {
  return v.p == nullptr || (((uintptr_t)v.p % (4 * esz)) == 0 && v.sb % 4 == 0 && v.st % 4 == 0);
}

// A segment's offsets in an array are 31-bit, with the tiles fetched ahead.
// Where time strides are too long for the plan's segments, *steps becomes what
// they allow, and time goes in windows of that many, one launch after another.
int stride_steps(const View &v, int esz, int *steps) {
  if (!v.p || v.st == 0) return PR_OK;
  if (v.st < 0) return fail(PR_EUNSUPPORTED, "time stride %lld is negative", v.st);
  const long long most = v.st > 2147483000LL / (9 * SSM_TL * esz) ? 0 : 2147483000LL / (v.st * esz) - 8 * SSM_TL;
  if (most < SSM_TL)
    return fail(PR_EUNSUPPORTED, "time stride %lld: at most %lld elements", v.st, 2147483000LL / (9 * SSM_TL * esz));
  if (most < *steps) *steps = (int)(most / SSM_TL * SSM_TL);
  return PR_OK;
}

int ssm_fill(const pr_ssm_problem *p, const SsmPlan &pl, const pr_ssm_inputs *in, SsmArgs *a, int *steps) {
  if (!in) return fail(PR_EINVAL, "inputs are NULL");
  if (!in->u.p || !in->dt.p || !in->B.p || !in->C.p || !in->A) return fail(PR_EINVAL, "u, dt, A, B and C are required");
  a->u = view(&in->u, p->T); a->dt = view(&in->dt, p->T); a->z = view(&in->z, p->T);
  a->Bm = view(&in->B, p->T); a->Cm = view(&in->C, p->T);
  a->A = in->A; a->Dk = in->D; a->bias = in->dt_bias; a->h0 = in->h0; a->lengths = in->lengths;
  a->B = p->B; a->T = p->T; a->D = p->D; a->N = p->N; a->G = p->G; a->softplus = p->softplus != 0;
  a->dpg = p->D / p->G; a->cbg = pl.cbg;
  const int esz = p->dtype == PR_BF16 ? 2 : 4;
  // a lane's states are there or not as a whole: eight of them from 33 states on
  a->vec = a->dpg % 4 == 0 && p->N % (p->N > 32 ? 8 : 4) == 0 && vec4_ok(a->u, esz) && vec4_ok(a->dt, esz) && vec4_ok(a->z, esz) &&
           vec4_ok(a->Bm, esz) && vec4_ok(a->Cm, esz);
  int rc = PR_OK;
  for (const View *v : {&a->u, &a->dt, &a->z, &a->Bm, &a->Cm})
    if ((rc = stride_steps(*v, esz, steps)) != PR_OK) return rc;
  if (p->N % 4 == 0 && (((uintptr_t)in->A | (uintptr_t)in->h0) & 15))
    return fail(PR_EINVAL, "A and h0 must be 16-byte aligned");
  return PR_OK;
}

int launch_ssm(int dtype, const SsmArgs &a, int what, hipStream_t s) {
  const hipError_t e = dtype == PR_BF16 ? (a.vec ? launch_ssm_bf16_vec(a, what, s) : launch_ssm_bf16(a, what, s))
                                        : (a.vec ? launch_ssm_f32_vec(a, what, s) : launch_ssm_f32(a, what, s));
  if (e != hipSuccess) return fail(PR_EHIP, "selective scan kernel: %s", hipGetErrorString(e));
  return PR_OK;
}

int check_ws(const void *ws, size_t have, size_t need) {
  if (!ws || have < need) return fail(PR_EWORKSPACE, "workspace %zu bytes < %zu", have, need);
  if (((uintptr_t)ws & 255) != 0) return fail(PR_EINVAL, "workspace must be 256-byte aligned");
  return PR_OK;
}

template <bool REV>
int join(const SsmArgs &a, const float *first, hipStream_t s) {
  const long long n = (long long)a.B * a.D * a.N;
  k_ssm_join<REV><<<flat_grid((n + 255) / 256), 256, 0, s>>>(a.A, first, a.sumd, a.agg, a.B, a.D, a.N, a.SA);
  HIPCHK(hipGetLastError());
  return PR_OK;
}

// Time in windows of `steps` steps: no segments side by side, one state per
// sequence (which the join kernel fills) goes from launch to launch.
void windows(SsmArgs *a, int steps) {
  a->S = a->R = a->SA = 1;
  a->seglen = steps;
  a->carry = a->agg;
}

}  // namespace

extern "C" {

size_t pararnn_ssm_workspace_bytes(const pr_ssm_problem *p, int with_adjoint) {
  clear_error();
  SsmPlan pl;
  if (ssm_plan(p, &pl) != PR_OK) return 0;
  return with_adjoint ? pl.adj_bytes : pl.fwd_bytes;
}

int pararnn_ssm_scan(const pr_ssm_problem *p, const pr_ssm_inputs *in, const pr_view *y, float *h_last, float *states,
                     void *workspace, size_t ws_bytes, void *stream) {
  clear_error();
  SsmPlan pl;
  int rc = ssm_plan(p, &pl);
  if (rc != PR_OK) return rc;
  SsmArgs a{};
  int steps = pl.seglen;
  rc = ssm_fill(p, pl, in, &a, &steps);
  if (rc != PR_OK) return rc;
  if (!y || !y->p) return fail(PR_EINVAL, "y is required");
  rc = check_ws(workspace, ws_bytes, pl.fwd_bytes);
  if (rc != PR_OK) return rc;
  a.y = view(y, p->T);
  if ((rc = stride_steps(a.y, p->dtype == PR_BF16 ? 2 : 4, &steps)) != PR_OK) return rc;
  a.vec = a.vec && vec4_ok(a.y, p->dtype == PR_BF16 ? 2 : 4);
  a.hlast = h_last; a.states = states;
  if (p->N % 4 == 0 && (((uintptr_t)h_last | (uintptr_t)states) & 15))
    return fail(PR_EINVAL, "h_last and states must be 16-byte aligned");
  char *ws = (char *)workspace;
  a.agg = (float *)(ws + pl.off_agg); a.sumd = (float *)(ws + pl.off_sumd);
  a.S = pl.S; a.seglen = pl.seglen; a.R = pl.R; a.SA = pl.S * pl.R;
  hipStream_t s = (hipStream_t)stream;
  if (steps < pl.seglen) {
    windows(&a, steps);
    if ((rc = join<false>(a, a.h0, s)) != PR_OK) return rc;
    for (a.win = 0; (long long)a.win * steps < p->T; a.win++)
      if ((rc = launch_ssm(p->dtype, a, SSM_FWD, s)) != PR_OK) return rc;
    return PR_OK;
  }
  if (a.S > 1) {
    if ((rc = launch_ssm(p->dtype, a, SSM_FWD_AGG, s)) != PR_OK) return rc;
    if ((rc = join<false>(a, a.h0, s)) != PR_OK) return rc;
  }
  return launch_ssm(p->dtype, a, SSM_FWD, s);
}

int pararnn_ssm_adjoint(const pr_ssm_problem *p, const pr_ssm_inputs *in, const float *states, const pr_view *dy,
                        const float *dh_last, const pr_ssm_grads *gr, void *workspace, size_t ws_bytes, void *stream) {
  clear_error();
  SsmPlan pl;
  int rc = ssm_plan(p, &pl);
  if (rc != PR_OK) return rc;
  SsmArgs a{};
  int steps = pl.seglen;
  rc = ssm_fill(p, pl, in, &a, &steps);
  if (rc != PR_OK) return rc;
  if (!states || !dy || !dy->p || !gr) return fail(PR_EINVAL, "states, dy and the gradients' struct are required");
  if (gr->z.p && !in->z.p) return fail(PR_EINVAL, "dz without z");
  rc = check_ws(workspace, ws_bytes, pl.adj_bytes);
  if (rc != PR_OK) return rc;
  const int esz = p->dtype == PR_BF16 ? 2 : 4;
  a.states = (float *)states; a.dhlast = dh_last; a.dh0 = gr->h0;
  a.dy = view(dy, p->T); a.du = view(&gr->u, p->T); a.ddt = view(&gr->dt, p->T); a.dz = view(&gr->z, p->T);
  a.dB = view(&gr->B, p->T); a.dC = view(&gr->C, p->T);
  for (const View *v : {&a.dy, &a.du, &a.ddt, &a.dz})
    if ((rc = stride_steps(*v, esz, &steps)) != PR_OK) return rc;
  a.vec = a.vec && vec4_ok(a.dy, esz) && vec4_ok(a.du, esz) && vec4_ok(a.ddt, esz) && vec4_ok(a.dz, esz);
  if (p->N % 4 == 0 && (((uintptr_t)states | (uintptr_t)dh_last | (uintptr_t)gr->h0) & 15))
    return fail(PR_EINVAL, "states, dh_last and dh0 must be 16-byte aligned");
  char *ws = (char *)workspace;
  a.agg = (float *)(ws + pl.off_agg); a.sumd = (float *)(ws + pl.off_sumd);
  a.part = (float *)(ws + pl.off_part); a.pA = (float *)(ws + pl.off_pA); a.pD = (float *)(ws + pl.off_pD);
  a.acc = (float *)(ws + pl.off_acc);
  a.S = pl.S; a.seglen = pl.seglen; a.R = pl.R; a.SA = pl.S * pl.R;
  hipStream_t s = (hipStream_t)stream;
  if (steps < pl.seglen) {
    windows(&a, steps);
    if ((rc = join<true>(a, dh_last, s)) != PR_OK) return rc;
    for (a.win = (p->T - 1) / steps; a.win >= 0; a.win--) {
      if ((rc = launch_ssm(p->dtype, a, SSM_ADJ, s)) != PR_OK) return rc;
      a.accum = 1;
    }
  } else {
    if (a.S > 1) {
      if ((rc = launch_ssm(p->dtype, a, SSM_ADJ_AGG, s)) != PR_OK) return rc;
      if ((rc = join<true>(a, dh_last, s)) != PR_OK) return rc;
    }
    if ((rc = launch_ssm(p->dtype, a, SSM_ADJ, s)) != PR_OK) return rc;
  }
  SsmSums f{};
  f.part = a.part; f.pA = a.pA; f.pD = a.pD; f.lengths = a.lengths; f.dB = a.dB; f.dC = a.dC;
  f.dA = gr->A; f.dD = gr->D; f.dbias = gr->dt_bias;
  f.nblk = a.cbg; f.B = a.B; f.T = a.T; f.G = a.G; f.N = a.N; f.NP = pl.NP; f.P = a.B * a.S; f.D = a.D;
  // a thread for each output, up to what one grid dimension takes beside the other kinds
  const long long bc = ((long long)a.B * a.T * a.G * 2 * pl.NP + 255) / 256;
  if (a.dB.p || a.dC.p) f.bc_blocks = (unsigned)(bc < (1 << 23) ? bc : 1 << 23);
  if (gr->A) f.a_blocks = (unsigned)(((long long)a.D * a.N + 31) / 32);
  const unsigned n = f.bc_blocks + f.a_blocks + (gr->D || gr->dt_bias ? 2 * ((a.D + 31) / 32) : 0);
  if (n == 0) return PR_OK;
  if (p->dtype == PR_BF16) k_ssm_sums<uint16_t><<<dim3(n), 256, 0, s>>>(f);
  else k_ssm_sums<float><<<dim3(n), 256, 0, s>>>(f);
  HIPCHK(hipGetLastError());
  return PR_OK;
}

int pararnn_ssm_step(const pr_ssm_problem *p, const pr_ssm_inputs *in, const pr_view *y, float *state, int nslots,
                     const int *slots, void *stream) {
  clear_error();
  const int rc = ssm_check(p, true);
  if (rc != PR_OK) return rc;
  if (p->B > 65535) return fail(PR_EUNSUPPORTED, "B = %d: at most 65535", p->B);
  if (!in) return fail(PR_EINVAL, "inputs are NULL");
  if (!in->u.p || !in->dt.p || !in->B.p || !in->C.p || !in->A || !y || !y->p || !state)
    return fail(PR_EINVAL, "u, dt, A, B, C, y and the states are required");
  if (nslots < 1 || (!slots && nslots < p->B)) return fail(PR_EINVAL, "%d states for %d sequences", nslots, p->B);
  if (p->N % 4 == 0 && (((uintptr_t)state | (uintptr_t)in->A) & 15))
    return fail(PR_EINVAL, "A and the states must be 16-byte aligned");
  SsmStepArgs a{};
  a.u = in->u.p; a.dt = in->dt.p; a.z = in->z.p; a.Bm = in->B.p; a.Cm = in->C.p; a.y = y->p;
  a.su = in->u.sb; a.sdt = in->dt.sb; a.sz = in->z.sb; a.sB = in->B.sb; a.sC = in->C.sb; a.sy = y->sb;
  a.A = in->A; a.Dk = in->D; a.bias = in->dt_bias; a.state = state; a.slots = slots;
  a.B = p->B; a.D = p->D; a.N = p->N; a.G = p->G; a.nslots = nslots; a.softplus = p->softplus != 0;
  HIPCHK(p->dtype == PR_BF16 ? launch_step<uint16_t>(a, (hipStream_t)stream) : launch_step<float>(a, (hipStream_t)stream));
  return PR_OK;
}

}  // extern "C"
