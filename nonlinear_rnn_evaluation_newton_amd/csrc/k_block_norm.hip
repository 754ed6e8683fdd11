// Norms around a block, joined with its gate and the residual's scale:
//   u = x rstd(x) w scale act(z),  t = residual + u,  y = t rstd(t) w_next
// and the adjoint, from the stored t (x^ = x rstd1, t^ = t rstd2):
//   gt = dt + rstd2 (w_next dy - t^ mean(w_next dy t^)),  dresidual = gt
//   e = gt w scale act(z),  dx = rstd1 (e - x^ mean(e x^)),
//   dz = gt w scale x^ act'(z),  q = sum over rows of gt act(z) x^,
//   dw = scale q,  dscale = w q,  dw_next = sum over rows of dy t^
//
// Bound by memory: every array is read or written once while a row stays in
// registers, 16 bytes a thread and access.  Between a block's two norms nothing goes
// through memory but t.  Squares and dot products are summed in fp32, the weights'
// gradients over the rows in fp32 within a block and in fp64 over the blocks.
// Measured, 16384 x 2048, bf16, with gate and residual: forward 57 us for 336 MB (in
// part from the last-level cache; VALU issue 84% by the counters), adjoint 106 us for 550
// MB (5.2 TB/s, 77%), the weights' sums 8; the same in fp32 on 8192 rows 160 together.
// Instructions count as much as bytes here: with a division by n and a square root for
// each sum, and row addresses in vector registers, a pass took 166 us for 161 to 163.
// Widths that do not fill the threads take more: 20000 x 1111 with a gate 126 us (52 at
// the rate of a copy), in fp32 143 (103); 4096 x 8192 with both 178 (130).
#include "pararnn.h"
#include "ssm.h"
#include "vec.h"

namespace pr {

struct BnArgs {
  const void *x, *z, *res, *w, *scale, *wn, *dt, *dy;  // z, res, w, scale, wn, dt, dy may be null
  void *t, *y, *dx, *dz, *dres;                        // the last four may be null
  float *stat;   // adjoint, long rows: [rows][3], rstd1, rstd2, rstd2^2 mean(w_next dy t)
  float *part;   // adjoint: partials of q | dw_next, [parts][2][n]
  long long lx, lz, lres, lt, ly, ldt, ldy, ldx, ldz, ldres;  // row strides
  long long rows;
  int n, gate;
  float eps, nf, rn;  // n and 1 / n
};

// sum / n to the nearest: the product with the rounded 1 / n, corrected by its exact
// remainder.  (An infinite sum has none.)
__device__ inline float mean_of(float sum, const BnArgs &a) {
  const float q = sum * a.rn, c = fmaf(fmaf(-q, a.nf, sum), a.rn, q);
  return c == c ? c : q;
}
// 1 / sqrt(mean + eps) to the nearest (but for values next to a tie): the hardware's
// instruction, good to one place, with one Newton step on its exact remainder.  It takes
// no denormals, and of 0 and infinity its own answer stands.
__device__ inline float rstd_of(float sum, const BnArgs &a) {
  const float v0 = mean_of(sum, a) + a.eps;
  const bool small = v0 < 0x1p-96f;
  const float v = small ? v0 * 0x1p64f : v0, y = __builtin_amdgcn_rsqf(v);
  const float h = v * y, l = fmaf(v, y, -h), e = fmaf(-l, y, fmaf(-h, y, 1.f)), c = fmaf(0.5f * y, e, y);
  return (c == c ? c : y) * (small ? 0x1p32f : 1.f);
}

// sigm(z).  A plain product as the exponential's argument is off by |z| 2^-24 of the
// result: far below a step of rows stored in 8 significant bits, but not of fp32 ones.
template <typename T>
__device__ inline float sigm_of(float z) {
  return sizeof(T) == 2 ? fsigm(z) : frcp(1.f + exp_any(-z));
}
// act(z) and its derivative from p = sigm(z): both are a factor, z or a number,
// of p and of p (1 - p), plus p times a number.  The gate's kind is the same for a
// whole launch: one select, so that no branch stands between the loads of a row.
struct Gate {
  bool silu;
  float k, c;  // act = (silu ? z : k) p; without a gate z is 0 and act = 2 sigm(0)
  __device__ Gate(const void *z, int kind) : silu(z && kind == PR_GATE_SILU), k(z ? 1.f : 2.f), c(silu ? 1.f : 0.f) {}
};
__device__ inline float act_of(const Gate &g, float z, float p) { return (g.silu ? z : g.k) * p; }
__device__ inline float act_d(const Gate &g, float z, float p) {
  return fmaf(g.silu ? z : g.k, p * (1.f - p), g.c * p);
}
template <typename T>
__device__ inline float act_v(const Gate &g, float z) { return act_of(g, z, sigm_of<T>(z)); }
template <typename T>
__device__ inline float to_storage(float v) {
  T t;
  stf(&t, 0, v);
  return ldf(&t, 0);
}
template <typename T>
__device__ inline float at1(const void *p, long long i) {
  return p ? ldf((const T *)p, i) : 1.f;
}

// Sum over a block of 256, the same in all threads, in a fixed order.  Calls
// one after another alternate between the halves of `sh`.
__device__ inline float block_sum(float v, float *sh) {
  v = wave_total(v);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  return (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

// Rows that stay in registers: TPR threads a row, NV vectors of V elements (16
// bytes) a thread.  EDGE: n is no multiple of V, and a row's last vector is its
// last V elements, of which the first `dup` belong to the vector before: they are
// left out of the sums, and not written (a result may stand where an input did
// that the other thread has still to read).
template <typename T>
constexpr int bn_v() { return 16 / (int)sizeof(T); }
struct BnAt {
  int c, dup;  // first element, or -1; elements that another thread counts
};
template <typename T, int TPR, bool EDGE>
__device__ inline BnAt bn_at(int x, int m, int n) {
  constexpr int V = bn_v<T>();
  const int c = (x + m * TPR) * V;
  if (c >= n) return BnAt{-1, EDGE ? V : 0};
  if (EDGE && c > n - V) return BnAt{n - V, c - (n - V)};
  return BnAt{c, 0};
}
template <typename T>
__device__ inline VecU<T, bn_v<T>()> bn_ld(const void *p, long long row, long long ld, const BnAt &at, bool there) {
  return ldu<T, bn_v<T>()>((const T *)p + row * ld + at.c, there && at.c >= 0 ? bn_v<T>() : 0);
}
template <typename T, bool EDGE>
__device__ inline void bn_st(void *p, long long row, long long ld, const BnAt &at, const float *f) {
  constexpr int V = bn_v<T>();
  T *o = (T *)p + row * ld + at.c;
  if (!EDGE || at.dup == 0) {
    if (at.c >= 0) stu_nt<T, V>(o, f, V);
  } else {
#pragma unroll
    for (int i = 1; i < V; i++)
      if (i >= at.dup) stf(o, i, f[i]);
  }
}
// N sums over the threads of a row, the same in all of them, in a fixed order;
// rows of several wavefronts use one half of sh for each call, in turn.
template <int TPR, int N>
__device__ inline void row_sums(float (&v)[N], float (*sh)[16]) {
#pragma unroll
  for (int k = 0; k < N; k++) v[k] = wave_total(v[k]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < N; k++) sh[k][threadIdx.x >> 6] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; k++) {
      float s = sh[k][0];
#pragma unroll
      for (int w = 1; w < W; w++) s += sh[k][w];
      v[k] = s;
    }
  }
}

template <typename T, int TPR, int NV, bool EDGE>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void k_bn(BnArgs a) {
  constexpr int V = bn_v<T>(), RPB = TPR > 256 ? 1 : 256 / TPR;
  __shared__ float sh[2][1][16];
  const int x = threadIdx.x % TPR;
  const long long row = flat_block() * RPB + __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  if (row >= a.rows) return;  // whole wavefronts, whole rows
  VecU<T, V> vx[NV], vz[NV], vr[NV];
  float ss[1] = {0.f};
#pragma unroll
  for (int m = 0; m < NV; m++) {
    const BnAt at = bn_at<T, TPR, EDGE>(x, m, a.n);
    vx[m] = bn_ld<T>(a.x, row, a.lx, at, true);
    vz[m] = bn_ld<T>(a.z, row, a.lz, at, a.z != nullptr);
    vr[m] = bn_ld<T>(a.res, row, a.lres, at, a.res != nullptr);
  }
  // (read while the row is on its way: the compiler would put these loads behind it)
  asm volatile("" : "+s"(a.eps), "+s"(a.nf), "+s"(a.rn), "+s"(a.gate), "+s"(a.lt), "+s"(a.ly));
  VecU<T, V> vw[NV], vs[NV], vn[NV];
#pragma unroll
  for (int m = 0; m < NV; m++) {
    const BnAt at = bn_at<T, TPR, EDGE>(x, m, a.n);
    vw[m] = bn_ld<T>(a.w, 0, 0, at, a.w != nullptr);
    vs[m] = bn_ld<T>(a.scale, 0, 0, at, a.scale != nullptr);
    vn[m] = bn_ld<T>(a.wn, 0, 0, at, a.y && a.wn);
#pragma unroll
    for (int i = 0; i < V; i++) {
      const float v = vx[m].f(i);
      ss[0] = !EDGE || i >= at.dup ? fmaf(v, v, ss[0]) : ss[0];
    }
  }
  row_sums<TPR, 1>(ss, sh[0]);
  const float rstd = rstd_of(ss[0], a);
  const Gate gate(a.z, a.gate);
  ss[0] = 0.f;
  float t[NV][V];
#pragma unroll
  for (int m = 0; m < NV; m++) {
    const BnAt at = bn_at<T, TPR, EDGE>(x, m, a.n);
#pragma unroll
    for (int i = 0; i < V; i++) {
      const float u = vx[m].f(i) * rstd * ((a.w ? vw[m].f(i) : 1.f) * (a.scale ? vs[m].f(i) : 1.f)) * act_v<T>(gate, vz[m].f(i));
      t[m][i] = to_storage<T>(a.res ? vr[m].f(i) + u : u);
      ss[0] = !EDGE || i >= at.dup ? fmaf(t[m][i], t[m][i], ss[0]) : ss[0];
    }
    bn_st<T, EDGE>(a.t, row, a.lt, at, t[m]);
  }
  if (!a.y) return;
  row_sums<TPR, 1>(ss, sh[1]);
  const float rstd2 = rstd_of(ss[0], a);
#pragma unroll
  for (int m = 0; m < NV; m++) {
    const BnAt at = bn_at<T, TPR, EDGE>(x, m, a.n);
#pragma unroll
    for (int i = 0; i < V; i++) t[m][i] *= rstd2 * (a.wn ? vn[m].f(i) : 1.f);
    bn_st<T, EDGE>(a.y, row, a.ly, at, t[m]);
  }
}

// The adjoint on rows in registers.  One round of sums for a row: with
// F = w scale act(z) x, sum(e x) = sum(dt F) + rstd2 (sum(w_next dy F) - k2 sum(t F)),
// k2 = rstd2^2 mean(w_next dy t).  Blocks walk rows with a stride of the grid and
// keep their columns' sums in registers, and where a row is at most two vectors a
// thread its weights in fp32 and each gate's sigmoid too.  Longer rows are loaded
// again, from cache, once their sums are known: there are no registers for them.
template <typename T, int TPR, int NV, bool EDGE>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256, NV == 1 ? 3 : 2) void k_bn_adj(BnArgs a) {
  constexpr int V = bn_v<T>(), RPB = TPR > 256 ? 1 : 256 / TPR, NT = TPR > 256 ? TPR : 256;
  constexpr bool AGAIN = NV > 2;
  __shared__ float sh[2][6][16];
  const int x = threadIdx.x % TPR, sub = __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
  int xr = x;
  const Gate gate(a.z, a.gate);
  float q[NV][V], qn[NV][V];
  float F[NV][V], wn[NV][V];  // w scale, w_next
  auto weights = [&](int m) __attribute__((always_inline)) {
    const BnAt at = bn_at<T, TPR, EDGE>(xr, m, a.n);
    const VecU<T, V> vw = bn_ld<T>(a.w, 0, 0, at, a.w != nullptr), vs = bn_ld<T>(a.scale, 0, 0, at, a.scale != nullptr),
                     vn = bn_ld<T>(a.wn, 0, 0, at, a.wn != nullptr);
#pragma unroll
    for (int i = 0; i < V; i++) {
      F[m][i] = (a.w ? vw.f(i) : 1.f) * (a.scale ? vs.f(i) : 1.f);
      wn[m][i] = a.wn ? vn.f(i) : 1.f;
    }
  };
#pragma unroll
  for (int m = 0; m < NV; m++) {
    if constexpr (!AGAIN) weights(m);
#pragma unroll
    for (int i = 0; i < V; i++) q[m][i] = qn[m][i] = 0.f;
  }
  int par = 0;
  for (long long row = (long long)blockIdx.x * RPB + sub; row < a.rows; row += (long long)gridDim.x * RPB) {
    VecU<T, V> vx[NV], vz[NV], vt[NV], vd[NV], vy[NV];
    float pz[AGAIN ? 1 : NV][V];
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto load = [&](int m) __attribute__((always_inline)) {
      const BnAt at = bn_at<T, TPR, EDGE>(xr, m, a.n);
      vx[m] = bn_ld<T>(a.x, row, a.lx, at, true);
      vz[m] = bn_ld<T>(a.z, row, a.lz, at, a.z != nullptr);
      vt[m] = bn_ld<T>(a.t, row, a.lt, at, a.dy != nullptr);
      vy[m] = bn_ld<T>(a.dy, row, a.ldy, at, a.dy != nullptr);
      vd[m] = bn_ld<T>(a.dt, row, a.ldt, at, a.dt != nullptr);
    };
    if constexpr (!AGAIN)
#pragma unroll
      for (int m = 0; m < NV; m++) load(m);
#pragma unroll
    for (int m = 0; m < NV; m++) {
      const BnAt at = bn_at<T, TPR, EDGE>(xr, m, a.n);
      if constexpr (AGAIN) {
        asm volatile("" : "+v"(xr) : : "memory");  // (one vector's loads at a time)
        weights(m);
        load(m);
      }
#pragma unroll
      for (int i = 0; i < V; i++) {
        const float p = sigm_of<T>(vz[m].f(i));
        if constexpr (!AGAIN) pz[m][i] = p;
        if (EDGE && i < at.dup) continue;
        const float xx = vx[m].f(i), t = vt[m].f(i), e = wn[m][i] * vy[m].f(i);
        const float f = F[m][i] * act_of(gate, vz[m].f(i), p) * xx;
        s[0] = fmaf(xx, xx, s[0]);
        s[1] = fmaf(vd[m].f(i), f, s[1]);
        s[2] = fmaf(t, t, s[2]);
        s[3] = fmaf(e, t, s[3]);
        s[4] = fmaf(e, f, s[4]);
        s[5] = fmaf(t, f, s[5]);
      }
    }
    row_sums<TPR, 6>(s, sh[par]);
    par ^= 1;  // the next row's sums go to the other half
    const float rstd1 = rstd_of(s[0], a), rstd2 = a.dy ? rstd_of(s[2], a) : 0.f;  // without dy: t and dy are zeros
    const float k2 = mean_of(s[3], a) * rstd2 * rstd2;
    const float k1 = mean_of(s[1] + rstd2 * (s[4] - k2 * s[5]), a) * rstd1 * rstd1;
#pragma unroll
    for (int m = 0; m < NV; m++) {
      const BnAt at = bn_at<T, TPR, EDGE>(xr, m, a.n);
      float ox[V], oz[V], og[V];
      if constexpr (AGAIN) {
        asm volatile("" : "+v"(xr) : : "memory");  // (one vector's loads at a time)
        weights(m);
        load(m);
      } else {  // (as they were stored: unpacked they would take twice the registers)
        asm volatile("" : "+v"(vx[m].v), "+v"(vz[m].v), "+v"(vt[m].v), "+v"(vd[m].v), "+v"(vy[m].v));
      }
#pragma unroll
      for (int i = 0; i < V; i++) {
        const float x_ = vx[m].f(i), xh = x_ * rstd1, t = vt[m].f(i), dy = vy[m].f(i), z = vz[m].f(i);
        const float p = AGAIN ? sigm_of<T>(z) : pz[AGAIN ? 0 : m][i], act = act_of(gate, z, p);
        const float g = fmaf(rstd2, fmaf(-t, k2, wn[m][i] * dy), vd[m].f(i)), gf = g * F[m][i];
        qn[m][i] = fmaf(dy, t * rstd2, qn[m][i]);
        q[m][i] = fmaf(g * act, xh, q[m][i]);
        og[i] = g;
        oz[i] = gf * xh * act_d(gate, z, p);
        ox[i] = rstd1 * fmaf(-x_, k1, gf * act);
      }
      if (a.dres) bn_st<T, EDGE>(a.dres, row, a.ldres, at, og);
      if (a.dz) bn_st<T, EDGE>(a.dz, row, a.ldz, at, oz);
      if (a.dx) bn_st<T, EDGE>(a.dx, row, a.ldx, at, ox);
    }
  }
  if (!a.part) return;
  float *pp = a.part + blockIdx.x * 2LL * a.n;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int m = 0; m < NV; m++) {
      const BnAt at = bn_at<T, TPR, EDGE>(x, m, a.n);
#pragma unroll
      for (int i = 0; i < V; i += 4)
        if (at.c >= 0 && at.dup == 0) {
          stu<float, 4>(pp + at.c + i, q[m] + i, 4);
          stu<float, 4>(pp + a.n + at.c + i, qn[m] + i, 4);
        }
      if (EDGE && at.c >= 0 && at.dup > 0)
#pragma unroll
        for (int i = 1; i < V; i++)
          if (i >= at.dup) {
            pp[at.c + i] = q[m][i];
            pp[a.n + at.c + i] = qn[m][i];
          }
    }
  } else {  // join the block's rows
    __shared__ float red[RPB][NV * V * TPR];
#pragma unroll
    for (int k = 0; k < 2; k++) {
      __syncthreads();
#pragma unroll
      for (int m = 0; m < NV; m++) {
        const BnAt at = bn_at<T, TPR, EDGE>(x, m, a.n);
#pragma unroll
        for (int i = 0; i < V; i++)
          if (at.c >= 0 && i >= at.dup) red[sub][at.c + i] = k ? qn[m][i] : q[m][i];
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.n; c += NT) {
        float v = red[0][c];
#pragma unroll
        for (int m = 1; m < RPB; m++) v += red[m][c];
        pp[(long long)k * a.n + c] = v;
      }
    }
  }
}

// N sums over a row's n elements, a thread's share of them: in fp32 over 256 elements
// at a time, which 64 bits join.  (One fp32 sum of a long row's squares drops the small
// ones as it grows: the gradients of 2^26 elements were off by 5e-5 to 3e-4.)
template <int N, typename F>
__device__ inline void long_sums(int n, float (&out)[N], F add) {
  constexpr int PIECE = 256 * 256;
  double total[N] = {};
  for (int c0 = threadIdx.x; c0 < n; c0 += PIECE) {
    const int c1 = n - c0 < PIECE ? n : c0 + PIECE;
    float s[N] = {};
    for (int c = c0; c < c1; c += 256) add(c, s);
#pragma unroll
    for (int k = 0; k < N; k++) total[k] += (double)s[k];
  }
#pragma unroll
  for (int k = 0; k < N; k++) out[k] = (float)total[k];
}

// Long rows (more than 16384 values of bf16 or 8192 of fp32; the adjoint's of bf16 more
// than 12288) and rows shorter than a vector: a block reads its row again, from
// cache, for each pass, element by element.
template <typename T>
__global__ __launch_bounds__(256) void k_bn_long(BnArgs a) {
  __shared__ float sh[2][4];
  const long long row = flat_block();
  if (row >= a.rows) return;
  const T *xp = (const T *)a.x + row * a.lx, *zp = (const T *)a.z + row * a.lz, *rp = (const T *)a.res + row * a.lres;
  T *tp = (T *)a.t + row * a.lt;
  const Gate gate(a.z, a.gate);
  float ss[1];
  long_sums(a.n, ss, [&](int c, float (&s)[1]) {
    const float v = ldf(xp, c);
    s[0] = fmaf(v, v, s[0]);
  });
  const float rstd = rstd_of(block_sum(ss[0], sh[0]), a);
  long_sums(a.n, ss, [&](int c, float (&s)[1]) {
    float u = ldf(xp, c) * rstd * (at1<T>(a.w, c) * at1<T>(a.scale, c));
    if (a.z) u *= act_v<T>(gate, ldf(zp, c));
    const float t = to_storage<T>(a.res ? ldf(rp, c) + u : u);
    stf(tp, c, t);
    s[0] = fmaf(t, t, s[0]);
  });
  if (!a.y) return;
  const float rstd2 = rstd_of(block_sum(ss[0], sh[1]), a);
  for (int c = threadIdx.x; c < a.n; c += 256)
    stf((T *)a.y + row * a.ly, c, ldf(tp, c) * rstd2 * at1<T>(a.wn, c));
}

// What a row's values give once its sums are known.
struct BnRow {
  float rstd1, rstd2, k2;  // k2 = rstd2^2 mean(w_next dy t)
};
template <typename T>
__device__ inline float bn_gt(const BnArgs &a, const BnRow &s, long long row, int c) {
  float g = a.dt ? ldf((const T *)a.dt + row * a.ldt, c) : 0.f;
  if (a.dy)
    g += s.rstd2 * fmaf(-ldf((const T *)a.t + row * a.lt, c), s.k2,
                        at1<T>(a.wn, c) * ldf((const T *)a.dy + row * a.ldy, c));
  return g;
}
template <typename T>
__global__ __launch_bounds__(256) void k_bn_adj_stat(BnArgs a) {
  __shared__ float sh[3][4];
  const long long row = flat_block();
  if (row >= a.rows) return;
  float sums[3];
  long_sums(a.n, sums, [&](int c, float (&s)[3]) {
    const float v = ldf((const T *)a.x + row * a.lx, c);
    s[0] = fmaf(v, v, s[0]);
    if (a.dy) {
      const float t = ldf((const T *)a.t + row * a.lt, c);
      s[1] = fmaf(t, t, s[1]);
      s[2] = fmaf(at1<T>(a.wn, c) * ldf((const T *)a.dy + row * a.ldy, c), t, s[2]);
    }
  });
  const float ss = block_sum(sums[0], sh[0]), st = block_sum(sums[1], sh[1]), dot = block_sum(sums[2], sh[2]);
  if (threadIdx.x == 0) {
    float *o = a.stat + row * 3;
    const float rstd2 = rstd_of(st, a);
    o[0] = rstd_of(ss, a);
    o[1] = rstd2;
    o[2] = mean_of(dot, a) * rstd2 * rstd2;
  }
}
// q and dw_next: a block sums one slice of the rows for 256 columns
template <typename T>
__global__ __launch_bounds__(256) void k_bn_adj_cols(BnArgs a, int slices) {
  const int cb = (a.n + 255) / 256, c = (int)(flat_block() % cb) * 256 + threadIdx.x;
  const long long slice = flat_block() / cb;
  if (slice >= slices || c >= a.n) return;
  const long long per = (a.rows + slices - 1) / slices, r0 = slice * per;
  const long long r1 = r0 + per < a.rows ? r0 + per : a.rows;
  const Gate gate(a.z, a.gate);
  float q = 0.f, wn = 0.f;
  for (long long r = r0; r < r1; r++) {
    const BnRow s{a.stat[r * 3], a.stat[r * 3 + 1], a.stat[r * 3 + 2]};
    const float xh = ldf((const T *)a.x + r * a.lx, c) * s.rstd1;
    const float act = a.z ? act_v<T>(gate, ldf((const T *)a.z + r * a.lz, c)) : 1.f;
    q = fmaf(bn_gt<T>(a, s, r, c) * act, xh, q);
    if (a.dy)
      wn = fmaf(ldf((const T *)a.dy + r * a.ldy, c), ldf((const T *)a.t + r * a.lt, c) * s.rstd2, wn);
  }
  a.part[slice * 2 * a.n + c] = q;
  a.part[(slice * 2 + 1) * a.n + c] = wn;
}
template <typename T>
__global__ __launch_bounds__(256) void k_bn_adj_long(BnArgs a) {
  __shared__ float sh[4];
  const long long row = flat_block();
  if (row >= a.rows) return;
  const BnRow s{a.stat[row * 3], a.stat[row * 3 + 1], a.stat[row * 3 + 2]};
  const T *xp = (const T *)a.x + row * a.lx, *zp = (const T *)a.z + row * a.lz;
  const Gate gate(a.z, a.gate);
  float dot[1];
  long_sums(a.n, dot, [&](int c, float (&v)[1]) {
    float e = bn_gt<T>(a, s, row, c) * (at1<T>(a.w, c) * at1<T>(a.scale, c));
    if (a.z) e *= act_v<T>(gate, ldf(zp, c));
    v[0] = fmaf(e, ldf(xp, c), v[0]);
  });
  const float k1 = mean_of(block_sum(dot[0], sh), a) * s.rstd1 * s.rstd1;
  for (int c = threadIdx.x; c < a.n; c += 256) {
    const float gt = bn_gt<T>(a, s, row, c), ws = at1<T>(a.w, c) * at1<T>(a.scale, c), x = ldf(xp, c);
    const float z = a.z ? ldf(zp, c) : 0.f, p = sigm_of<T>(z);
    if (a.dres) stf((T *)a.dres + row * a.ldres, c, gt);
    if (a.dz) stf((T *)a.dz + row * a.ldz, c, gt * ws * (x * s.rstd1) * act_d(gate, z, p));
    if (a.dx) stf((T *)a.dx + row * a.ldx, c, s.rstd1 * fmaf(-x, k1, gt * ws * act_of(gate, z, p)));
  }
}

// The weights' gradients from the partials [P][2][n], in 64 bits in a fixed
// order: 16 columns by 64 slices of the partials a block.
template <typename T>
__global__ __launch_bounds__(1024) void k_bn_sums(const float *__restrict__ part, int P, int n, const void *w,
                                                  const void *scale, float *dw, float *dscale, float *dwn) {
  __shared__ double sh[64][17];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4, k = blockIdx.z;
  const long long c = flat_block() * 16 + x;
  if (k ? !dwn : !dw && !dscale) return;
  double s = 0;
  if (c < n)
    for (int p0 = y; p0 < P; p0 += 512) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; q++) v[q] = p0 + 64 * q < P ? part[((p0 + 64LL * q) * 2 + k) * n + c] : 0.f;
#pragma unroll
      for (int q = 0; q < 8; q++) s += (double)v[q];
    }
  sh[y][x] = s;
  for (int h = 32; h >= 1; h >>= 1) {
    __syncthreads();
    if (y < h) sh[y][x] += sh[y + h][x];
  }
  if (y != 0 || c >= n) return;
  const float v = (float)sh[0][x];
  if (k) {
    dwn[c] = v;
  } else {
    if (dw) dw[c] = v * at1<T>(scale, c);
    if (dscale) dscale[c] = v * at1<T>(w, c);
  }
}

// Threads and vectors of a row of q vectors; 0 threads: the row is read again
// for each pass.  The adjoint holds five inputs and two sums: two vectors a thread
// stay in registers, and four of fp32 rows or three of bf16 ones are loaded twice.
struct BnGeom {
  int tpr, nv;
};
static BnGeom bn_geom(int n, int V, bool adj) {
  if (n < V) return {0, 0};
  const int q = (n + V - 1) / V;
  if (q <= 64) return {64, 1};
  if (q <= 128) return {64, 2};
  if (q <= 256) return {256, 1};
  if (q <= 512) return {256, 2};
  if (q <= 1024) return adj ? BnGeom{512, 2} : BnGeom{256, 4};
  if (adj && V == 8) return q <= 1536 ? BnGeom{512, 3} : BnGeom{0, 0};
  if (q <= 2048) return {512, 4};
  return {0, 0};
}

// (FOR_ADJ: the geometry is the adjoint's or the forward's alone; -1: both's)
template <typename T, int TPR, int NV, int FOR_ADJ = -1>
void bn_go(const BnArgs &a, bool adj, unsigned blocks, hipStream_t s) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  const bool edge = a.n % bn_v<T>() != 0;
  const dim3 rows = flat_grid((a.rows + NT / TPR - 1) / (NT / TPR));
  if constexpr (FOR_ADJ != 0)
    if (adj) {
      if (edge) k_bn_adj<T, TPR, NV, true><<<blocks, NT, 0, s>>>(a);
      else k_bn_adj<T, TPR, NV, false><<<blocks, NT, 0, s>>>(a);
    }
  if constexpr (FOR_ADJ != 1)
    if (!adj) {
      if (edge) k_bn<T, TPR, NV, true><<<rows, NT, 0, s>>>(a);
      else k_bn<T, TPR, NV, false><<<rows, NT, 0, s>>>(a);
    }
}
template <typename T>
hipError_t bn_launch(const BnArgs &a, const BnGeom &g, bool adj, unsigned blocks, hipStream_t s) {
  if (g.tpr == 64 && g.nv == 1) bn_go<T, 64, 1>(a, adj, blocks, s);
  else if (g.tpr == 64) bn_go<T, 64, 2>(a, adj, blocks, s);
  else if (g.tpr == 256 && g.nv == 1) bn_go<T, 256, 1>(a, adj, blocks, s);
  else if (g.tpr == 256 && g.nv == 2) bn_go<T, 256, 2>(a, adj, blocks, s);
  else if (g.tpr == 256) bn_go<T, 256, 4, false>(a, adj, blocks, s);
  else if (g.nv == 2) bn_go<T, 512, 2, true>(a, adj, blocks, s);
  else if (!adj) bn_go<T, 512, 4, false>(a, adj, blocks, s);
  else bn_go<T, 512, sizeof(T) == 2 ? 3 : 4, true>(a, adj, blocks, s);
  return hipGetLastError();
}

}  // namespace pr

using namespace pr;

namespace {

#define HIPCHK(expr)                                                                        \
  do {                                                                                      \
    hipError_t e_ = (expr);                                                                 \
    if (e_ != hipSuccess) return fail(PR_EHIP, "%s: %s", #expr, hipGetErrorString(e_));     \
  } while (0)

constexpr int BN_SLICES = 64;  // slices of the rows in the columns' sums of long rows
// The most rows that a thread adds in fp32, 2^-25 of the sum lost at each: more rows are
// more partials, which 64 bits add (from 32768 long rows on, from 131072 wide ones, from
// a million short ones).
constexpr int BN_ROWS = 512;

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
bool has(const pr_rows *r) { return r && r->p; }

int bn_check(const pr_block_norm_problem *p) {
  if (!p) return fail(PR_EINVAL, "problem is NULL");
  if (p->dtype != PR_F32 && p->dtype != PR_BF16) return fail(PR_EINVAL, "unknown dtype %d", p->dtype);
  if (p->rows < 1 || p->n < 1) return fail(PR_EINVAL, "sizes must be >= 1 (rows=%lld n=%d)", p->rows, p->n);
  if (!(p->eps >= 0.f) || p->eps > 3.0e38f) return fail(PR_EINVAL, "eps must be >= 0 and finite");
  if (p->rows > 2147483647LL || p->n > (1 << 30)) return fail(PR_EUNSUPPORTED, "problem too large");
  return PR_OK;
}

int bn_fill(const pr_block_norm_problem *p, const pr_rows *x, const pr_rows *z, const void *w, const void *scale,
            const void *wn, BnArgs *a) {
  if (!has(x)) return fail(PR_EINVAL, "x is required");
  a->x = x->p; a->lx = x->ld;
  if (has(z)) {
    if (p->gate != PR_GATE_SILU && p->gate != PR_GATE_SIGMOID) return fail(PR_EINVAL, "unknown gate %d", p->gate);
    a->z = z->p; a->lz = z->ld;
  }
  a->w = w; a->scale = scale; a->wn = wn;
  a->rows = p->rows; a->n = p->n; a->gate = p->gate; a->eps = p->eps; a->nf = (float)p->n; a->rn = 1.f / a->nf;
  return PR_OK;
}

struct BnPlan {
  BnGeom g;
  size_t off_part, bytes;
  int parts;
};
BnPlan bn_plan(const pr_block_norm_problem *p) {
  BnPlan pl;
  pl.g = bn_geom(p->n, p->dtype == PR_BF16 ? 8 : 4, true);
  size_t o = 0;
  if (pl.g.tpr) {
    // as many blocks of bf16 rows as run at once on 256 CUs (by the kernels' registers 3
    // wavefronts a SIMD with one vector, 2 with more), each with its share of the rows:
    // with more, the last ones run on a device that is half empty, and there are more
    // partials.  Of fp32 rows 4 and 3 where 5 and 4 would fit, which was not compared.
    // (The workspace's size is asked for without a device too: a count of 256 CUs.)
    const long long rpb = pl.g.tpr > 256 ? 1 : 256 / pl.g.tpr, b = (p->rows + rpb - 1) / rpb;
    const int per_simd = (p->dtype == PR_BF16 ? 2 : 3) + (pl.g.nv == 1 ? 1 : 0);
    const long long most = 256 * (pl.g.tpr > 256 ? 1 : per_simd);
    const long long least = (b + BN_ROWS - 1) / BN_ROWS;
    pl.parts = (int)(b < most ? b : least < most ? most : least);
  } else {
    const long long least = (p->rows + BN_ROWS - 1) / BN_ROWS;
    pl.parts = (int)(p->rows < BN_SLICES ? p->rows : least < BN_SLICES ? BN_SLICES : least);
    o = align256((size_t)p->rows * 12);
  }
  pl.off_part = o;
  pl.bytes = align256(o + (size_t)pl.parts * 2 * p->n * 4);
  return pl;
}

}  // namespace

extern "C" {

int pararnn_block_norm(const pr_block_norm_problem *p, const pr_rows *x, const pr_rows *z, const pr_rows *residual,
                       const void *w, const void *scale, const void *w_next, const pr_rows *t, const pr_rows *y,
                       void *stream) {
  clear_error();
  int rc = bn_check(p);
  if (rc != PR_OK) return rc;
  BnArgs a{};
  if ((rc = bn_fill(p, x, z, w, scale, w_next, &a)) != PR_OK) return rc;
  if (!has(t)) return fail(PR_EINVAL, "t is required");
  a.t = t->p; a.lt = t->ld;
  if (has(residual)) { a.res = residual->p; a.lres = residual->ld; }
  if (has(y)) { a.y = y->p; a.ly = y->ld; }
  hipStream_t s = (hipStream_t)stream;
  const BnGeom g = bn_geom(p->n, p->dtype == PR_BF16 ? 8 : 4, false);
  if (g.tpr) {
    HIPCHK(p->dtype == PR_BF16 ? bn_launch<uint16_t>(a, g, false, 0, s) : bn_launch<float>(a, g, false, 0, s));
    return PR_OK;
  }
  const dim3 grid = flat_grid(p->rows);
  if (p->dtype == PR_BF16) k_bn_long<uint16_t><<<grid, 256, 0, s>>>(a);
  else k_bn_long<float><<<grid, 256, 0, s>>>(a);
  HIPCHK(hipGetLastError());
  return PR_OK;
}

size_t pararnn_block_norm_workspace_bytes(const pr_block_norm_problem *p) {
  clear_error();
  if (bn_check(p) != PR_OK) return 0;
  return bn_plan(p).bytes;
}

int pararnn_block_norm_adjoint(const pr_block_norm_problem *p, const pr_rows *x, const pr_rows *z, const void *w,
                               const void *scale, const void *w_next, const pr_rows *t, const pr_rows *dt,
                               const pr_rows *dy, const pr_block_norm_grads *gr, void *workspace, size_t ws_bytes,
                               void *stream) {
  clear_error();
  int rc = bn_check(p);
  if (rc != PR_OK) return rc;
  BnArgs a{};
  if ((rc = bn_fill(p, x, z, w, scale, w_next, &a)) != PR_OK) return rc;
  if (!gr) return fail(PR_EINVAL, "the gradients' struct is required");
  if (!has(dt) && !has(dy)) return fail(PR_EINVAL, "one of dt and dy is required");
  if (has(dy) && !has(t)) return fail(PR_EINVAL, "dy without t");
  if (gr->z.p && !has(z)) return fail(PR_EINVAL, "dz without z");
  if (gr->w_next && !has(dy)) return fail(PR_EINVAL, "dw_next without dy");
  const BnPlan pl = bn_plan(p);
  if (!workspace || ws_bytes < pl.bytes) return fail(PR_EWORKSPACE, "workspace %zu bytes < %zu", ws_bytes, pl.bytes);
  if (((uintptr_t)workspace & 255) != 0) return fail(PR_EINVAL, "workspace must be 256-byte aligned");
  if (has(t)) { a.t = t->p; a.lt = t->ld; }
  if (has(dt)) { a.dt = dt->p; a.ldt = dt->ld; }
  if (has(dy)) { a.dy = dy->p; a.ldy = dy->ld; }
  a.dx = gr->x.p; a.ldx = gr->x.ld; a.dz = gr->z.p; a.ldz = gr->z.ld; a.dres = gr->res.p; a.ldres = gr->res.ld;
  char *ws = (char *)workspace;
  const bool bf = p->dtype == PR_BF16, sums = gr->w || gr->scale || gr->w_next;
  float *part = (float *)(ws + pl.off_part);
  hipStream_t s = (hipStream_t)stream;
  if (pl.g.tpr) {
    a.part = sums ? part : nullptr;
    HIPCHK(bf ? bn_launch<uint16_t>(a, pl.g, true, (unsigned)pl.parts, s)
              : bn_launch<float>(a, pl.g, true, (unsigned)pl.parts, s));
  } else {
    a.stat = (float *)ws;
    a.part = part;
    const dim3 grid = flat_grid(p->rows), cols = flat_grid(((long long)p->n + 255) / 256 * pl.parts);
    if (bf) k_bn_adj_stat<uint16_t><<<grid, 256, 0, s>>>(a);
    else k_bn_adj_stat<float><<<grid, 256, 0, s>>>(a);
    HIPCHK(hipGetLastError());
    if (sums) {  // before the rows' gradients, of which dres may stand over dt
      if (bf) k_bn_adj_cols<uint16_t><<<cols, 256, 0, s>>>(a, pl.parts);
      else k_bn_adj_cols<float><<<cols, 256, 0, s>>>(a, pl.parts);
      HIPCHK(hipGetLastError());
    }
    if (a.dx || a.dz || a.dres) {
      if (bf) k_bn_adj_long<uint16_t><<<grid, 256, 0, s>>>(a);
      else k_bn_adj_long<float><<<grid, 256, 0, s>>>(a);
      HIPCHK(hipGetLastError());
    }
  }
  if (!sums) return PR_OK;
  dim3 grid = flat_grid(((long long)p->n + 15) / 16);
  grid.z = 2;
  if (bf) k_bn_sums<uint16_t><<<grid, 1024, 0, s>>>(part, pl.parts, p->n, w, scale, gr->w, gr->scale, gr->w_next);
  else k_bn_sums<float><<<grid, 1024, 0, s>>>(part, pl.parts, p->n, w, scale, gr->w, gr->scale, gr->w_next);
  HIPCHK(hipGetLastError());
  return PR_OK;
}

}  // extern "C"
