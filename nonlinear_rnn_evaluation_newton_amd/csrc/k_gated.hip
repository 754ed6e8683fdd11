// Gated linear recurrence, its adjoint and its single-token step.
//
//   r = sigm(rg + rb), i = sigm(ig + ib), v = decay r, a = e^-v,
//   m = sqrt(1 - a^2), h_t = a h_{t-1} + m i x_t
// Adjoint, with g_t = dy_t + a_{t+1} g_{t+1}:
//   dx = g m i, di = g m x i (1 - i), dv = g (a^2 / m i x - a h_{t-1}),
//   dr = dv decay r (1 - r), ddecay = sum dv r
#include "pararnn.h"
#include "ssm.h"
#include "vec.h"

namespace pr {

struct GatedArgs {
  View x, r, i, y;           // y: the output, or dy in the adjoint
  View dx, dr, di;           // adjoint; may be null
  const float *decay, *rb, *ib, *h0;  // rb, ib, h0 may be null
  const int *lengths;        // may be null
  float *hlast, *states;     // may be null (states is required by the adjoint)
  const float *dhlast;       // adjoint, may be null
  float *dh0;                // adjoint, may be null
  float *part;               // adjoint: partials of ddecay | dr_bias | di_bias, [part][3][D]
  int B, T, D;
};

constexpr int GS = 128;  // steps between two saved states

// What a step's gates give: a = e^-v and 1 - a^2 for v = decay r, both gates
// and their complements.
struct GateVals {
  float r, r1, i, i1, a, m2;
};
template <typename T>
__device__ inline float gate_exp(float x) {
  if constexpr (sizeof(T) == 2) return fexp(x);
  else return exp_acc(x);
}
template <typename T>
__device__ inline GateVals gate_vals(float rg, float ig, float decay) {
  GateVals o;
  const float er = gate_exp<T>(-rg), ei = gate_exp<T>(-ig);
  o.r = frcp(1.f + er);
  o.i = frcp(1.f + ei);
  // 1 - sigm = e sigm keeps the digits of a gate that is nearly open (where e
  // is infinite the product is NaN, which the minimum drops)
  o.r1 = fminf(er * o.r, 1.f);
  o.i1 = fminf(ei * o.i, 1.f);
  const float v = decay * o.r;
  o.a = gate_exp<T>(-v);
  // 1 - e^-w for w = 2 v: the difference where little is lost, else its series
  // (the first term left out is below w^6 / 5040 of it, 5e-8 at w = 1/4)
  const float w = v + v;
  float s = fmaf(w, -1.f / 720.f, 1.f / 120.f);
  s = fmaf(w, s, -1.f / 24.f);
  s = fmaf(w, s, 1.f / 6.f);
  s = fmaf(w, s, -0.5f);
  s = fmaf(w, s, 1.f);
  o.m2 = w < 0.25f ? w * s : fmaf(-o.a, o.a, 1.f);
  return o;
}
constexpr float GATE_TINY = 1.17549435e-38f;  // 1 - a^2 below it counts as 0

// One thread per (sequence, channel) through all steps.
template <typename T>
__global__ __launch_bounds__(64) void k_gated_fwd(GatedArgs a) {
  const long long id = flat_block() * 64 + threadIdx.x;
  if (id >= (long long)a.B * a.D) return;
  const int d = (int)(id % a.D), b = (int)(id / a.D);
  const int len = seq_len(a.lengths, b, a.T);
  const float decay = a.decay[d], rb = a.rb ? a.rb[d] : 0.f, ib = a.ib ? a.ib[d] : 0.f;
  float h = a.h0 ? a.h0[id] : 0.f;
  const int nst = (a.T + GS - 1) / GS;
  for (int t = 0; t < a.T; t++) {
    if (t < len) {
      if (a.states && t % GS == 0) a.states[((long long)b * nst + t / GS) * a.D + d] = h;
      const GateVals g = gate_vals<T>(ldf((const T *)a.r.p, b * a.r.sb + t * a.r.st + d) + rb,
                                      ldf((const T *)a.i.p, b * a.i.sb + t * a.i.st + d) + ib, decay);
      const float m = g.m2 >= GATE_TINY ? __builtin_amdgcn_sqrtf(g.m2) : 0.f;
      h = fmaf(g.a, h, m * g.i * ldf((const T *)a.x.p, b * a.x.sb + t * a.x.st + d));
    }
    stf((T *)a.y.p, b * a.y.sb + t * a.y.st + d, t < len ? h : 0.f);
  }
  if (a.hlast) a.hlast[id] = h;
}

// The same back in time: the states of 16 steps at a time are made again from
// the saved one.
template <typename T>
__global__ __launch_bounds__(64) void k_gated_adj(GatedArgs a) {
  const long long id = flat_block() * 64 + threadIdx.x;
  if (id >= (long long)a.B * a.D) return;
  const int d = (int)(id % a.D), b = (int)(id / a.D);
  const int len = seq_len(a.lengths, b, a.T);
  const float decay = a.decay[d], rb = a.rb ? a.rb[d] : 0.f, ib = a.ib ? a.ib[d] : 0.f;
  const int nst = (a.T + GS - 1) / GS;
  float mu = a.dhlast ? a.dhlast[id] : 0.f, sv = 0.f, sr = 0.f, si = 0.f;
  auto vals = [&](int t, float *x) {
    *x = ldf((const T *)a.x.p, b * a.x.sb + t * a.x.st + d);
    return gate_vals<T>(ldf((const T *)a.r.p, b * a.r.sb + t * a.r.st + d) + rb,
                        ldf((const T *)a.i.p, b * a.i.sb + t * a.i.st + d) + ib, decay);
  };
  for (int t0 = (a.T - 1) / 16 * 16; t0 >= 0; t0 -= 16) {
    float hp[16];
    const int c0 = t0 / GS * GS;
    float h = c0 < len ? a.states[((long long)b * nst + c0 / GS) * a.D + d] : 0.f;
    for (int t = c0; t < t0 + 16; t++) {
      if (t >= t0) {
#pragma unroll
        for (int k = 0; k < 16; k++)
          if (t == t0 + k) hp[k] = h;
      }
      if (t < len) {
        float x;
        const GateVals g = vals(t, &x);
        h = fmaf(g.a, h, (g.m2 >= GATE_TINY ? __builtin_amdgcn_sqrtf(g.m2) : 0.f) * g.i * x);
      }
    }
#pragma unroll
    for (int k = 15; k >= 0; k--) {
      const int t = t0 + k;
      if (t >= a.T) continue;
      float ox = 0.f, orr = 0.f, oi = 0.f;
      if (t < len) {
        float x;
        const GateVals g = vals(t, &x);
        const float rm = g.m2 >= GATE_TINY ? __builtin_amdgcn_rsqf(g.m2) : 0.f, m = g.m2 * rm;
        const float gg = mu + ldf((const T *)a.y.p, b * a.y.sb + t * a.y.st + d);
        const float gi = gg * g.i;
        ox = gi * m;
        oi = ox * x * g.i1;
        const float dv = g.a * fmaf(gi * x, g.a * rm, -gg * hp[k]);
        sv = fmaf(dv, g.r, sv);
        orr = dv * decay * g.r * g.r1;
        sr += orr;
        si += oi;
        mu = gg * g.a;
      }
      if (a.dx.p) stf((T *)a.dx.p, b * a.dx.sb + t * a.dx.st + d, ox);
      if (a.dr.p) stf((T *)a.dr.p, b * a.dr.sb + t * a.dr.st + d, orr);
      if (a.di.p) stf((T *)a.di.p, b * a.di.sb + t * a.di.st + d, oi);
    }
  }
  if (a.dh0) a.dh0[id] = mu;
  if (a.part) {
    float *p = a.part + (long long)b * 3 * a.D + d;
    p[0] = sv;
    p[a.D] = sr;
    p[2LL * a.D] = si;
  }
}

struct GatedStepArgs {
  const void *x, *r, *i;
  void *y;
  long long sx, sr, si, sy;
  const float *decay, *rb, *ib;
  float *state;
  const int *slots;
  int B, D, nslots;
};

// One token: four channels a thread.
template <typename T>
__global__ __launch_bounds__(256) void k_gated_step(GatedStepArgs a) {
  constexpr int V = 4;
  const int d = (int)(blockIdx.x * 256 + threadIdx.x) * V, b = blockIdx.y, n = a.D - d;
  if (n <= 0) return;
  const int slot = a.slots ? a.slots[b] : b;
  float o[V] = {0.f, 0.f, 0.f, 0.f};
  if (slot >= 0 && slot < a.nslots) {
    float *hp = a.state + (long long)slot * a.D + d;
    const VecU<T, V> x = ldu<T, V>((const T *)a.x + b * a.sx + d, n), r = ldu<T, V>((const T *)a.r + b * a.sr + d, n),
                     i = ldu<T, V>((const T *)a.i + b * a.si + d, n);
    const VecU<float, V> h = ldu<float, V>(hp, n), dc = ldu<float, V>(a.decay + d, n),
                         rb = ldu<float, V>(a.rb + d, a.rb ? n : 0), ib = ldu<float, V>(a.ib + d, a.ib ? n : 0);
#pragma unroll
    for (int k = 0; k < V; k++) {
      const GateVals g = gate_vals<T>(r.f(k) + rb.f(k), i.f(k) + ib.f(k), dc.f(k));
      const float m = g.m2 >= GATE_TINY ? __builtin_amdgcn_sqrtf(g.m2) : 0.f;
      o[k] = fmaf(g.a, h.f(k), m * g.i * x.f(k));
    }
    stu<float, V>(hp, o, n);
  }
  stu<T, V>((T *)a.y + b * a.sy + d, o, n);
}

}  // namespace pr

using namespace pr;

namespace {

#define HIPCHK(expr)                                                                        \
  do {                                                                                      \
    hipError_t e_ = (expr);                                                                 \
    if (e_ != hipSuccess) return fail(PR_EHIP, "%s: %s", #expr, hipGetErrorString(e_));     \
  } while (0)

// step: single tokens, T is not used and may be 0
int gated_check(const pr_gated_problem *p, bool step) {
  if (!p) return fail(PR_EINVAL, "problem is NULL");
  if (p->dtype != PR_F32 && p->dtype != PR_BF16) return fail(PR_EINVAL, "unknown dtype %d", p->dtype);
  if (p->B < 1 || p->T < (step ? 0 : 1) || p->D < 1)
    return fail(PR_EINVAL, "sizes must be >= 1 (B=%d T=%d D=%d)", p->B, p->T, p->D);
  if (p->T > (1 << 30)) return fail(PR_EUNSUPPORTED, "T = %d: at most 2^30", p->T);
  if (p->D > (1 << 24)) return fail(PR_EUNSUPPORTED, "D = %d: at most 2^24", p->D);
  return PR_OK;
}

struct GatedPlan {
  size_t fwd_bytes, adj_bytes;
};
int gated_plan(const pr_gated_problem *p, GatedPlan *pl) {
  const int rc = gated_check(p, false);
  if (rc != PR_OK) return rc;
  if ((double)p->B * p->T * p->D > 1e13) return fail(PR_EUNSUPPORTED, "problem too large");
  pl->fwd_bytes = 256;
  pl->adj_bytes = ((size_t)p->B * 3 * p->D * 4 + 255) & ~(size_t)255;
  return PR_OK;
}

View view(const pr_view *v) { return v && v->p ? View{v->p, v->sb, v->st} : View{nullptr, 0, 0}; }

int gated_fill(const pr_gated_problem *p, const pr_gated_inputs *in, GatedArgs *a) {
  if (!in) return fail(PR_EINVAL, "inputs are NULL");
  if (!in->x.p || !in->r.p || !in->i.p || !in->decay) return fail(PR_EINVAL, "x, r, i and decay are required");
  a->x = view(&in->x); a->r = view(&in->r); a->i = view(&in->i);
  a->decay = in->decay; a->rb = in->r_bias; a->ib = in->i_bias; a->h0 = in->h0; a->lengths = in->lengths;
  a->B = p->B; a->T = p->T; a->D = p->D;
  return PR_OK;
}

int check_ws(const void *ws, size_t have, size_t need) {
  if (!ws || have < need) return fail(PR_EWORKSPACE, "workspace %zu bytes < %zu", have, need);
  if (((uintptr_t)ws & 255) != 0) return fail(PR_EINVAL, "workspace must be 256-byte aligned");
  return PR_OK;
}

}  // namespace

extern "C" {

size_t pararnn_gated_workspace_bytes(const pr_gated_problem *p, int with_adjoint) {
  clear_error();
  GatedPlan pl;
  if (gated_plan(p, &pl) != PR_OK) return 0;
  return with_adjoint && pl.adj_bytes > pl.fwd_bytes ? pl.adj_bytes : pl.fwd_bytes;
}

int pararnn_gated_scan(const pr_gated_problem *p, const pr_gated_inputs *in, const pr_view *y, float *h_last,
                       float *states, void *workspace, size_t ws_bytes, void *stream) {
  clear_error();
  GatedPlan pl;
  int rc = gated_plan(p, &pl);
  if (rc != PR_OK) return rc;
  GatedArgs a{};
  if ((rc = gated_fill(p, in, &a)) != PR_OK) return rc;
  if (!y || !y->p) return fail(PR_EINVAL, "y is required");
  if ((rc = check_ws(workspace, ws_bytes, pl.fwd_bytes)) != PR_OK) return rc;
  a.y = view(y); a.hlast = h_last; a.states = states;
  hipStream_t s = (hipStream_t)stream;
  const dim3 grid = flat_grid(((long long)a.B * a.D + 63) / 64);
  if (p->dtype == PR_BF16) k_gated_fwd<uint16_t><<<grid, 64, 0, s>>>(a);
  else k_gated_fwd<float><<<grid, 64, 0, s>>>(a);
  HIPCHK(hipGetLastError());
  return PR_OK;
}

int pararnn_gated_adjoint(const pr_gated_problem *p, const pr_gated_inputs *in, const float *states, const pr_view *dy,
                          const float *dh_last, const pr_gated_grads *gr, void *workspace, size_t ws_bytes,
                          void *stream) {
  clear_error();
  GatedPlan pl;
  int rc = gated_plan(p, &pl);
  if (rc != PR_OK) return rc;
  GatedArgs a{};
  if ((rc = gated_fill(p, in, &a)) != PR_OK) return rc;
  if (!states || !dy || !dy->p || !gr) return fail(PR_EINVAL, "states, dy and the gradients' struct are required");
  if ((rc = check_ws(workspace, ws_bytes, pl.adj_bytes)) != PR_OK) return rc;
  a.y = view(dy); a.dx = view(&gr->x); a.dr = view(&gr->r); a.di = view(&gr->i);
  a.states = (float *)states; a.dhlast = dh_last; a.dh0 = gr->h0; a.h0 = nullptr;
  const bool sums = gr->decay || gr->r_bias || gr->i_bias;
  a.part = sums ? (float *)workspace : nullptr;
  hipStream_t s = (hipStream_t)stream;
  const dim3 grid = flat_grid(((long long)a.B * a.D + 63) / 64);
  if (p->dtype == PR_BF16) k_gated_adj<uint16_t><<<grid, 64, 0, s>>>(a);
  else k_gated_adj<float><<<grid, 64, 0, s>>>(a);
  HIPCHK(hipGetLastError());
  if (!sums) return PR_OK;
  float *out[3] = {gr->decay, gr->r_bias, gr->i_bias};
  for (int k = 0; k < 3; k++)
    if (out[k]) HIPCHK(launch_part_sum(a.part + (long long)k * a.D, a.B, 3LL * a.D, a.D, out[k], s));
  return PR_OK;
}

int pararnn_gated_step(const pr_gated_problem *p, const pr_gated_inputs *in, const pr_view *y, float *state, int nslots,
                       const int *slots, void *stream) {
  clear_error();
  const int rc = gated_check(p, true);
  if (rc != PR_OK) return rc;
  if (p->B > 65535) return fail(PR_EUNSUPPORTED, "B = %d: at most 65535", p->B);
  if (!in) return fail(PR_EINVAL, "inputs are NULL");
  if (!in->x.p || !in->r.p || !in->i.p || !in->decay || !y || !y->p || !state)
    return fail(PR_EINVAL, "x, r, i, decay, y and the states are required");
  if (nslots < 1 || (!slots && nslots < p->B)) return fail(PR_EINVAL, "%d states for %d sequences", nslots, p->B);
  GatedStepArgs a{};
  a.x = in->x.p; a.r = in->r.p; a.i = in->i.p; a.y = y->p;
  a.sx = in->x.sb; a.sr = in->r.sb; a.si = in->i.sb; a.sy = y->sb;
  a.decay = in->decay; a.rb = in->r_bias; a.ib = in->i_bias; a.state = state; a.slots = slots;
  a.B = p->B; a.D = p->D; a.nslots = nslots;
  const dim3 grid((unsigned)((p->D + 1023) / 1024), (unsigned)p->B);
  if (p->dtype == PR_BF16) k_gated_step<uint16_t><<<grid, 256, 0, (hipStream_t)stream>>>(a);
  else k_gated_step<float><<<grid, 256, 0, (hipStream_t)stream>>>(a);
  HIPCHK(hipGetLastError());
  return PR_OK;
}

}  // extern "C"
