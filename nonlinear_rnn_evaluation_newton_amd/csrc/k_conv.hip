// Short causal convolution per channel, its adjoint and its single-token step.
//
// Bound by memory: x is read and y written once.  A thread takes V adjacent
// channels (16 bytes where alignment allows) through a run of steps and keeps
// the last W - 1 inputs in registers, so a run re-reads only W - 1 steps.
// Measured (8 x 4096 x 2048, 4 taps; each kernel in calls one after another, and
// after 1 GiB of other writes): bf16 57 and 82 us, 4.7 and 3.3 TB/s, the adjoint
// 89 and 92 us, 4.5 TB/s, with four channels a lane (eight, and half the
// wavefronts: 116 to 110 us before the runs' own loop); fp32 94 and 128, the
// adjoint 178 us; its weights' sums 5 us; a step of 48 sequences 4 us, a launch.
#include <type_traits>

#include "pararnn.h"
#include "ssm.h"
#include "vec.h"

namespace pr {

struct ConvArgs {
  View x, y, dy, dx;
  const void *w, *bias, *sin, *dsout;
  void *sout, *dsin;
  const int *lengths;
  float *part;  // adjoint: [run blocks][W + 1][D]
  int B, T, D, silu;
  int run, runs;  // steps of a thread, runs per sequence
};

// The input of step t (t < 0: the state's) of channels d..
template <typename T, int V, int W>
__device__ inline VecOf<T, V> conv_in(const ConvArgs &a, int b, int t, int d, int len) {
  if (t >= 0) return ldv<T, V>((const T *)a.x.p + b * a.x.sb + t * a.x.st + d, t < len);
  return ldv<T, V>((const T *)a.sin + ((long long)b * (W - 1) + (t + W - 1)) * a.D + d, a.sin != nullptr);
}

template <typename T, int V, int W>
__device__ inline void conv_weights(const ConvArgs &a, int d, float (*w)[V], float *bias) {
#pragma unroll
  for (int i = 0; i < V; i++) {
#pragma unroll
    for (int k = 0; k < W; k++) w[k][i] = ldf((const T *)a.w, (size_t)(d + i) * W + k);
    bias[i] = a.bias ? ldf((const T *)a.bias, d + i) : 0.f;
  }
}

template <typename T, int V, int W>
__global__ __launch_bounds__(256) void k_conv_fwd(ConvArgs a) {
  const int nv = a.D / V, vb = (nv + 255) / 256;
  const unsigned blk = (unsigned)flat_block();
  const int d = ((int)(blk % vb) * 256 + threadIdx.x) * V;
  const int q = (int)(blk / vb), run = q % a.runs, b = q / a.runs;
  if (d >= a.D || b >= a.B) return;
  const int len = seq_len(a.lengths, b, a.T);
  const int t0 = run * a.run, t1 = a.T - t0 < a.run ? a.T : t0 + a.run;
  float w[W][V], bias[V], win[W][V];  // win[k]: the input of step t - W + 1 + k
  conv_weights<T, V, W>(a, d, w, bias);
#pragma unroll
  for (int k = 1; k < W; k++) {
    const VecOf<T, V> r = conv_in<T, V, W>(a, b, t0 - W + k, d, len);
#pragma unroll
    for (int i = 0; i < V; i++) win[k][i] = r.f(i);
  }
  if (run == 0 && a.sout) {  // reads the whole old state before it writes the new one
    VecOf<T, V> o[W];
#pragma unroll
    for (int k = 0; k < W - 1; k++) o[k] = conv_in<T, V, W>(a, b, len - (W - 1) + k, d, len);
#pragma unroll
    for (int k = 0; k < W - 1; k++)
      *reinterpret_cast<typename Vec<T, V>::type *>((T *)a.sout + ((long long)b * (W - 1) + k) * a.D + d) = o[k].v;
  }
  constexpr int U = 8;
  T *yp = (T *)a.y.p + b * a.y.sb + d;
  for (int t = t0; t < t1; t += U) {
    VecOf<T, V> in[U];
#pragma unroll
    for (int u = 0; u < U; u++)
      in[u] = ldv<T, V>((const T *)a.x.p + b * a.x.sb + (t + u) * a.x.st + d, t + u < t1 && t + u < len);
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (t + u >= t1) break;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; i++) {
#pragma unroll
        for (int k = 0; k < W - 1; k++) win[k][i] = win[k + 1][i];
        win[W - 1][i] = in[u].f(i);
        float s = bias[i];
#pragma unroll
        for (int k = 0; k < W; k++) s = fmaf(w[k][i], win[k][i], s);
        if (a.silu) s *= fsigm(s);
        o[i] = t + u < len ? s : 0.f;
      }
      stv<T, V>(yp + (t + u) * a.y.st, o);
    }
  }
}

// 64 channel vectors by 8 runs per block, a wavefront for each run, so that
// where it stands in its sequence is a scalar; dw and dbias of a block's runs
// are joined in shared memory in a fixed order.
template <typename T, int V, int W>
__global__ __launch_bounds__(512) void k_conv_adj(ConvArgs a) {
  __shared__ float red[8][W + 1][64 * V];
  const int nv = a.D / V, vb = (nv + 63) / 64;
  const int x = threadIdx.x & 63, r8 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned blk = (unsigned)flat_block();
  const int dblk = (int)(blk % vb) * 64, d = (dblk + x) * V;
  const long long q = (long long)(blk / vb) * 8 + r8;
  const bool on = d < a.D && q < (long long)a.B * a.runs;
  float gw[W][V], gb[V];
#pragma unroll
  for (int i = 0; i < V; i++) {
    gb[i] = 0.f;
#pragma unroll
    for (int k = 0; k < W; k++) gw[k][i] = 0.f;
  }
  if (on) {
    const int run = (int)(q % a.runs), b = (int)(q / a.runs);
    const int len = __builtin_amdgcn_readfirstlane(seq_len(a.lengths, b, a.T));
    const int t0 = run * a.run, t1 = a.T - t0 < a.run ? a.T : t0 + a.run;
    float w[W][V], bias[V], win[W][V], da[W][V];  // da[k]: of step t - W + 1 + k
    conv_weights<T, V, W>(a, d, w, bias);
#pragma unroll
    for (int k = 0; k < W; k++)
#pragma unroll
      for (int i = 0; i < V; i++) da[k][i] = win[k][i] = 0.f;
#pragma unroll
    for (int k = 1; k < W; k++) {
      const VecOf<T, V> r = conv_in<T, V, W>(a, b, t0 - W + k, d, len);
#pragma unroll
      for (int i = 0; i < V; i++) win[k][i] = r.f(i);
    }
    const bool own_state = run == 0;
    constexpr int U = 4;
    const T *xp = (const T *)a.x.p + b * a.x.sb + d, *gp = (const T *)a.dy.p + b * a.dy.sb + d;
    // Step tt: da there, its share of dw, and the input gradient of step
    // tt - W + 1, whose last tap it is.  FAST: tt and that step lie within the
    // run, and no gradient of the state reaches it.
    auto step = [&](auto fast, int tt, const VecOf<T, V> &in, const VecOf<T, V> &gy) __attribute__((always_inline)) {
      constexpr bool FAST = decltype(fast)::value;
      const bool own = FAST || tt < t1, live = FAST || tt < len;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; i++) {
#pragma unroll
        for (int k = 0; k < W - 1; k++) {
          win[k][i] = win[k + 1][i];
          da[k][i] = da[k + 1][i];
        }
        win[W - 1][i] = in.f(i);
        float s = bias[i];
#pragma unroll
        for (int k = 0; k < W; k++) s = fmaf(w[k][i], win[k][i], s);
        float g = gy.f(i);
        if (a.silu) {
          const float p = fsigm(s);
          g *= p * fmaf(s, 1.f - p, 1.f);
        }
        if (!live) g = 0.f;
        da[W - 1][i] = g;
        if (own && live) {
          gb[i] += g;
#pragma unroll
          for (int k = 0; k < W; k++) gw[k][i] = fmaf(g, win[k][i], gw[k][i]);
        }
        // the input of step tt - W + 1 meets tap W - 1 - k at step tt - W + 1 + k
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < W; k++) sum = fmaf(w[W - 1 - k][i], da[k][i], sum);
        o[i] = sum;
      }
      const int st = tt - (W - 1);
      if constexpr (FAST) {
        if (a.dx.p) stv<T, V>((T *)a.dx.p + b * a.dx.sb + st * a.dx.st + d, o);
      } else {
        const bool state_step = st < 0 && own_state;
        if (a.dsout && (st >= t0 || state_step) && st >= len - (W - 1) && st < len) {
          const VecOf<T, V> g =
              ldv<T, V>((const T *)a.dsout + ((long long)b * (W - 1) + st - (len - (W - 1))) * a.D + d, true);
#pragma unroll
          for (int i = 0; i < V; i++) o[i] += g.f(i);
        }
        if (st >= t0) {
          if (st >= len)
#pragma unroll
            for (int i = 0; i < V; i++) o[i] = 0.f;
          if (a.dx.p) stv<T, V>((T *)a.dx.p + b * a.dx.sb + st * a.dx.st + d, o);
        } else if (state_step && a.dsin) {
          stv<T, V>((T *)a.dsin + ((long long)b * (W - 1) + st + W - 1) * a.D + d, o);
        }
      }
    };
    // W - 1 steps past the run give the da that its last inputs still need;
    // the first run also walks back over the state's inputs
    int t = t0;
    const int slow = t0 + W - 1, fast_end = len < t1 ? len : t1;
    for (; t < slow && t < t1 + W - 1; t++) {
      const bool ok = t < len;
      const VecOf<T, V> in = ldv<T, V>(xp + t * a.x.st, ok), gy = ldv<T, V>(gp + t * a.dy.st, ok);
      step(std::integral_constant<bool, false>{}, t, in, gy);
    }
    for (; t + U <= fast_end; t += U) {
      VecOf<T, V> in[U], gy[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        in[u] = ldv<T, V>(xp + (t + u) * a.x.st, true);
        gy[u] = ldv<T, V>(gp + (t + u) * a.dy.st, true);
      }
#pragma unroll
      for (int u = 0; u < U; u++) step(std::integral_constant<bool, true>{}, t + u, in[u], gy[u]);
    }
    for (; t < t1 + W - 1; t++) {
      const bool ok = t < len;
      const VecOf<T, V> in = ldv<T, V>(xp + t * a.x.st, ok), gy = ldv<T, V>(gp + t * a.dy.st, ok);
      step(std::integral_constant<bool, false>{}, t, in, gy);
    }
  }
  if (!a.part || (long long)(blk / vb) * 8 >= (long long)a.B * a.runs) return;  // (past the end: a block as a whole)
#pragma unroll
  for (int i = 0; i < V; i++) {
#pragma unroll
    for (int k = 0; k < W; k++) red[r8][k][x * V + i] = gw[k][i];
    red[r8][W][x * V + i] = gb[i];
  }
  __syncthreads();
  float *o = a.part + (long long)(blk / vb) * (W + 1) * a.D;
  for (int i = threadIdx.x; i < (W + 1) * 64 * V; i += 512) {
    const int k = i / (64 * V), c = i % (64 * V), dd = dblk * V + c;
    if (dd < a.D) {
      float s = 0.f;
#pragma unroll
      for (int m = 0; m < 8; m++) s += red[m][k][c];
      o[(long long)k * a.D + dd] = s;
    }
  }
}

// dw [D][W] and dbias [D] from the blocks' partials, in 64 bits
__global__ void k_conv_wsum(const float *__restrict__ part, int P, int D, int W, float *dw, float *dbias) {
  __shared__ double sh[4][64];
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  const long long cols = (long long)(W + 1) * D, j = (long long)blockIdx.x * 64 + x;
  double s = 0;
  if (j < cols) {
#pragma unroll 4
    for (int p = y; p < P; p += 4) s += (double)part[p * cols + j];
  }
  sh[y][x] = s;
  __syncthreads();
  if (y == 0 && j < cols) {
    const float v = (float)((sh[0][x] + sh[1][x]) + (sh[2][x] + sh[3][x]));
    const int k = (int)(j / D), d = (int)(j % D);
    if (k == W) {
      if (dbias) dbias[d] = v;
    } else if (dw) {
      dw[(long long)d * W + k] = v;
    }
  }
}

struct ConvStepArgs {
  const void *x, *w, *bias;
  void *state, *y;
  long long sx, sy;
  const int *slots;
  int B, D, nslots, silu;
};

template <typename T, int V, int W>
__global__ __launch_bounds__(256) void k_conv_step(ConvStepArgs a) {
  const int d = (int)(blockIdx.x * 256 + threadIdx.x) * V, b = blockIdx.y;
  if (d >= a.D) return;
  const int slot = a.slots ? a.slots[b] : b;
  const bool live = slot >= 0 && slot < a.nslots;
  float o[V];
#pragma unroll
  for (int i = 0; i < V; i++) o[i] = 0.f;
  if (live) {
    VecOf<T, V> in[W];
    T *sp = (T *)a.state + (long long)slot * (W - 1) * a.D + d;
#pragma unroll
    for (int k = 0; k < W - 1; k++) in[k] = ldv<T, V>(sp + (long long)k * a.D, true);
    in[W - 1] = ldv<T, V>((const T *)a.x + b * a.sx + d, true);
#pragma unroll
    for (int i = 0; i < V; i++) {
      float s = a.bias ? ldf((const T *)a.bias, d + i) : 0.f;
#pragma unroll
      for (int k = 0; k < W; k++) s = fmaf(ldf((const T *)a.w, (size_t)(d + i) * W + k), in[k].f(i), s);
      if (a.silu) s *= fsigm(s);
      o[i] = s;
    }
#pragma unroll
    for (int k = 0; k < W - 1; k++)
      *reinterpret_cast<typename Vec<T, V>::type *>(sp + (long long)k * a.D) = in[k + 1].v;
  }
  stv<T, V>((T *)a.y + b * a.sy + d, o);
}

template <typename T, int V, int W>
hipError_t conv_fwd_launch(const ConvArgs &a, hipStream_t s) {
  const long long nv = a.D / V, q = (long long)a.B * a.runs;
  k_conv_fwd<T, V, W><<<flat_grid(((nv + 255) / 256) * q), 256, 0, s>>>(a);
  return hipGetLastError();
}
template <typename T, int V, int W>
hipError_t conv_adj_launch(const ConvArgs &a, hipStream_t s) {
  const long long nv = a.D / V, q = (long long)a.B * a.runs;
  k_conv_adj<T, V, W><<<flat_grid(((nv + 63) / 64) * ((q + 7) / 8)), 512, 0, s>>>(a);
  return hipGetLastError();
}
template <typename T, int V, int W>
hipError_t conv_step_launch(const ConvStepArgs &a, hipStream_t s) {
  k_conv_step<T, V, W><<<dim3((unsigned)((a.D / V + 255) / 256), (unsigned)a.B), 256, 0, s>>>(a);
  return hipGetLastError();
}

// f<T, V, W>() for the problem's storage, vector width and taps
#define PR_CONV_W(T, V, F, ...)                       \
  switch (W) {                                        \
    case 1: return F<T, V, 1>(__VA_ARGS__);           \
    case 2: return F<T, V, 2>(__VA_ARGS__);           \
    case 3: return F<T, V, 3>(__VA_ARGS__);           \
    default: return F<T, V, 4>(__VA_ARGS__);          \
  }
#define PR_CONV(V16, F, ...)                          \
  if (dtype == PR_BF16) {                             \
    if (vec) PR_CONV_W(uint16_t, V16, F, __VA_ARGS__) \
    PR_CONV_W(uint16_t, 1, F, __VA_ARGS__)            \
  }                                                   \
  if (vec) PR_CONV_W(float, 4, F, __VA_ARGS__)        \
  PR_CONV_W(float, 1, F, __VA_ARGS__)

static hipError_t conv_dispatch(int dtype, int W, bool vec, const ConvArgs &a, bool adj, hipStream_t s) {
  if (adj) {
    PR_CONV(4, conv_adj_launch, a, s)
  }
  PR_CONV(8, conv_fwd_launch, a, s)
}
static hipError_t conv_step_dispatch(int dtype, int W, bool vec, const ConvStepArgs &a, hipStream_t s) {
  PR_CONV(8, conv_step_launch, a, s)
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
int conv_check(const pr_conv_problem *p, bool step = false) {
  if (!p) return fail(PR_EINVAL, "problem is NULL");
  if (p->dtype != PR_F32 && p->dtype != PR_BF16) return fail(PR_EINVAL, "unknown dtype %d", p->dtype);
  if (p->B < 1 || p->T < (step ? 0 : 1) || p->D < 1 || p->W < 1)
    return fail(PR_EINVAL, "sizes must be >= 1 (B=%d T=%d D=%d W=%d)", p->B, p->T, p->D, p->W);
  if (p->W > 4) return fail(PR_EUNSUPPORTED, "W = %d taps: at most 4", p->W);
  if (p->T > (1 << 30)) return fail(PR_EUNSUPPORTED, "T = %d: at most 2^30", p->T);
  return PR_OK;
}

// Steps of a thread: long runs re-read little, short ones fill the device.
void conv_runs(const pr_conv_problem *p, int V, int *run, int *runs) {
  const long long lanes = (long long)p->B * ((p->D + V - 1) / V);
  int r = 64;
  while (r > 8 && lanes * ((p->T + r - 1) / r) < 4LL * 256 * 256) r >>= 1;
  *run = r;
  *runs = (p->T + r - 1) / r;
}

bool al16(const void *q) { return ((uintptr_t)q & 15) == 0; }
bool vecv_ok(const pr_view *v, int V) { return !v || !v->p || (al16(v->p) && v->sb % V == 0 && v->st % V == 0); }
View view(const pr_view *v) { return v ? View{v->p, v->sb, v->st} : View{nullptr, 0, 0}; }

}  // namespace

extern "C" {

size_t pararnn_conv_workspace_bytes(const pr_conv_problem *p) {
  clear_error();
  if (conv_check(p) != PR_OK) return 0;
  int run, runs;
  size_t most = 0;
  for (int V : {1, 4}) {
    conv_runs(p, V, &run, &runs);
    const size_t n = (((size_t)p->B * runs + 7) / 8) * (p->W + 1) * p->D * 4;
    most = n > most ? n : most;
  }
  return (most + 255) & ~(size_t)255;
}

int pararnn_conv(const pr_conv_problem *p, const pr_view *x, const void *w, const void *bias, const void *state_in,
                 const int *lengths, const pr_view *y, void *state_out, void *stream) {
  clear_error();
  int rc = conv_check(p);
  if (rc != PR_OK) return rc;
  if (!x || !x->p || !w || !y || !y->p) return fail(PR_EINVAL, "x, w and y are required");
  const int V = p->dtype == PR_BF16 ? 8 : 4;
  const bool vec = p->D % V == 0 && vecv_ok(x, V) && vecv_ok(y, V) && al16(state_in) && al16(state_out);
  ConvArgs a{};
  a.x = view(x); a.y = view(y); a.w = w; a.bias = bias; a.sin = state_in; a.sout = state_out; a.lengths = lengths;
  a.B = p->B; a.T = p->T; a.D = p->D; a.silu = p->silu != 0;
  conv_runs(p, vec ? V : 1, &a.run, &a.runs);
  if ((double)a.B * a.runs * (a.D / (vec ? V : 1) / 32 + 1) > 2e9) return fail(PR_EUNSUPPORTED, "problem too large");
  HIPCHK(conv_dispatch(p->dtype, p->W, vec, a, false, (hipStream_t)stream));
  return PR_OK;
}

int pararnn_conv_adjoint(const pr_conv_problem *p, const pr_view *x, const void *w, const void *bias,
                         const void *state_in, const int *lengths, const pr_view *dy, const void *dstate_out,
                         const pr_view *dx, float *dw, float *dbias, void *dstate_in, void *workspace,
                         size_t ws_bytes, void *stream) {
  clear_error();
  int rc = conv_check(p);
  if (rc != PR_OK) return rc;
  if (!x || !x->p || !w || !dy || !dy->p) return fail(PR_EINVAL, "x, w and dy are required");
  const size_t need = pararnn_conv_workspace_bytes(p);
  if (!workspace || ws_bytes < need) return fail(PR_EWORKSPACE, "workspace %zu bytes < %zu", ws_bytes, need);
  if (((uintptr_t)workspace & 255) != 0) return fail(PR_EINVAL, "workspace must be 256-byte aligned");
  const int V = 4;
  const bool vec = p->D % V == 0 && vecv_ok(x, V) && vecv_ok(dy, V) && vecv_ok(dx, V) && al16(state_in) &&
                   al16(dstate_out) && al16(dstate_in);
  ConvArgs a{};
  a.x = view(x); a.dy = view(dy); a.dx = view(dx); a.w = w; a.bias = bias; a.sin = state_in; a.dsout = dstate_out;
  a.dsin = dstate_in; a.lengths = lengths;
  a.B = p->B; a.T = p->T; a.D = p->D; a.silu = p->silu != 0;
  a.part = dw || dbias ? (float *)workspace : nullptr;
  conv_runs(p, vec ? V : 1, &a.run, &a.runs);
  if ((double)a.B * a.runs * (a.D / (vec ? V : 1) / 32 + 1) > 2e9) return fail(PR_EUNSUPPORTED, "problem too large");
  hipStream_t s = (hipStream_t)stream;
  HIPCHK(conv_dispatch(p->dtype, p->W, vec, a, true, s));
  if (a.part) {
    const int P = (int)(((long long)a.B * a.runs + 7) / 8);
    const long long cols = (long long)(p->W + 1) * p->D;
    k_conv_wsum<<<dim3((unsigned)((cols + 63) / 64)), 256, 0, s>>>(a.part, P, p->D, p->W, dw, dbias);
    HIPCHK(hipGetLastError());
  }
  return PR_OK;
}

int pararnn_conv_step(const pr_conv_problem *p, const pr_view *x, const void *w, const void *bias, void *state,
                      int nslots, const int *slots, const pr_view *y, void *stream) {
  clear_error();
  int rc = conv_check(p, true);
  if (rc != PR_OK) return rc;
  if (!x || !x->p || !w || !y || !y->p || (!state && p->W > 1)) return fail(PR_EINVAL, "x, w, state and y are required");
  if (nslots < 1 || (!slots && nslots < p->B)) return fail(PR_EINVAL, "%d states for %d sequences", nslots, p->B);
  if (p->B > 65535) return fail(PR_EUNSUPPORTED, "B = %d: at most 65535", p->B);
  const int V = p->dtype == PR_BF16 ? 8 : 4;
  const bool vec = p->D % V == 0 && al16(x->p) && x->sb % V == 0 && al16(y->p) && y->sb % V == 0 && al16(state);
  ConvStepArgs a{};
  a.x = x->p; a.w = w; a.bias = bias; a.state = state; a.y = y->p; a.sx = x->sb; a.sy = y->sb; a.slots = slots;
  a.B = p->B; a.D = p->D; a.nslots = nslots; a.silu = p->silu != 0;
  HIPCHK(conv_step_dispatch(p->dtype, p->W, vec, a, (hipStream_t)stream));
  return PR_OK;
}

}  // extern "C"
