// Root-mean-square norm with the residual's addition, in the storage type or
// in 8 bits with a scale for each row, its adjoint, and the 8-bit form of
// rows as they are.
//
// Bound by memory.  A row's values stay in registers between the sum of
// squares, the maximum and the output, so every array is read or written
// once: one wavefront holds a row of up to 64 x 4 vectors, a block one of up
// to 256 x 8; longer rows are read again (from cache) for each pass.  Squares are
// summed in fp32: a row whose sum overflows (values of 1e18 and more) gives y = 0.
// Measured (rows of 2048; calls one after another, whose inputs the last-level
// cache holds in part, and after 1 GiB of other writes): bf16 16384 rows with
// the residual 42 and 75 us, 8192 rows to 8 bits 20 and 36, the adjoint of 16384
// rows 45 and 48 and 7 us for the weight's sums, 16384 rows to 8 bits without a
// norm 17 and 31 (a wavefront has one row's loads in flight, then none while it
// reduces and stores); fp32 93 and 119, 32 and 64, 77 and 113, 24 and 52.  2048
// rows of 20000 in bf16, element by element: 104 and 136 us.
#include "pararnn.h"
#include "ssm.h"
#include "vec.h"

namespace pr {

enum { NORM_Y = 0, NORM_Q = 1, NORM_QUANT = 2 };  // storage out, 8 bits out, 8 bits without a norm

struct NormArgs {
  const void *x, *r, *w, *dy, *ds;
  void *s, *y, *dx;
  int8_t *q;
  float *scale, *part, *rstd;
  long long lx, lr, ls, ly, lq, ldy, lds, ldx;  // row strides
  long long rows;
  int n;
  float eps;
};

// Sum or maximum over the TPR threads of a row, the same in all of them, in a
// fixed order.  `sh` holds 4 floats; blocks of one row call it once per value
// with alternating halves.
template <int TPR>
__device__ inline float row_sum(float v, float *sh) {
  v = wave_total(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (sh[0] + sh[1]) + (sh[2] + sh[3]);
  }
  return v;
}
// of non-negative values; a NaN anywhere gives a NaN (its bits sort highest)
template <int TPR>
__device__ inline float row_max(float v, float *sh) {
  unsigned m = wave_max_dpp(__float_as_uint(v));
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = __uint_as_float(m);
    __syncthreads();
    m = max(max(__float_as_uint(sh[0]), __float_as_uint(sh[1])), max(__float_as_uint(sh[2]), __float_as_uint(sh[3])));
  }
  return __uint_as_float(m);
}

template <typename T>
__device__ inline float to_storage(float v) {
  T t;
  stf(&t, 0, v);
  return ldf(&t, 0);
}

// q = y / scale to the nearest, ties to even.  The quotient is the correctly
// rounded one (the product with a reciprocal alone would move values next to a
// tie): with inv the rounded reciprocal, the product's exact remainder times
// inv corrects it, three operations for a division's dozen.  Scales near the
// ends of the range are divided by.  A row with an infinity or a NaN is all 0:
// its scale carries that on.
template <int V>
__device__ inline void store_q(int8_t *p, const float *y, float scale) {
  VecOf<int8_t, V> o;
  const bool plain = scale > 1e-30f && scale < 1e30f;
  const float inv = plain ? __fdiv_rn(1.f, scale) : 0.f;
#pragma unroll
  for (int i = 0; i < V; i++) {
    float q;
    if (plain) {
      q = y[i] * inv;
      q = fmaf(fmaf(-q, scale, y[i]), inv, q);
    } else {
      q = scale > 0.f && scale < __builtin_inff() ? __fdiv_rn(y[i], scale) : 0.f;
    }
    o.e[i] = (int8_t)(int)fminf(fmaxf(rintf(q), -127.f), 127.f);
  }
  *reinterpret_cast<typename Vec<int8_t, V>::type *>(p) = o.v;
}

template <typename T, int V, int TPR, int NV, int MODE>
__global__ __launch_bounds__(256) void k_norm(NormArgs a) {
  constexpr int RPB = 256 / TPR;
  __shared__ float sh[2][4];
  const int x = threadIdx.x % TPR;
  const long long row = flat_block() * RPB + threadIdx.x / TPR;
  if (row >= a.rows) return;  // whole wavefronts, whole rows
  const T *xp = (const T *)a.x + row * a.lx, *rp = a.r ? (const T *)a.r + row * a.lr : nullptr;
  T *sp = a.s ? (T *)a.s + row * a.ls : nullptr;
  const T *wp = (const T *)a.w;
  constexpr int STEP = TPR * V;
  if constexpr (NV > 0) {
    float s[NV][V];
    VecOf<T, V> vx[NV], vr[NV], vw[NV];
#pragma unroll
    for (int m = 0; m < NV; m++) {
      const int c = x * V + m * STEP;
      vx[m] = ldv<T, V>(xp + c, c < a.n);
      if (MODE != NORM_QUANT && rp) vr[m] = ldv<T, V>(rp + c, c < a.n);
      if (MODE != NORM_QUANT && wp) vw[m] = ldv<T, V>(wp + c, c < a.n);
    }
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int m = 0; m < NV; m++) {
      const int c = x * V + m * STEP;
#pragma unroll
      for (int i = 0; i < V; i++) {
        float v = vx[m].f(i);
        if (MODE != NORM_QUANT && rp) v = to_storage<T>(v + vr[m].f(i));
        s[m][i] = v;
        if (MODE == NORM_QUANT) top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(fabsf(v))));
        else ss = fmaf(v, v, ss);
      }
      if (MODE != NORM_QUANT && sp && c < a.n) stv<T, V>(sp + c, s[m]);
    }
    if constexpr (MODE != NORM_QUANT) {
      ss = row_sum<TPR>(ss, sh[0]);
      const float rstd = 1.f / sqrtf(ss / (float)a.n + a.eps);
#pragma unroll
      for (int m = 0; m < NV; m++)
#pragma unroll
        for (int i = 0; i < V; i++) {
          s[m][i] = s[m][i] * rstd * (wp ? vw[m].f(i) : 1.f);
          if (MODE == NORM_Q) top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(fabsf(s[m][i]))));
        }
    }
    float scale = 0.f;
    if constexpr (MODE != NORM_Y) {
      scale = row_max<TPR>(top, sh[1]) * (1.f / 127.f);
      if (x == 0) a.scale[row] = scale;
    }
#pragma unroll
    for (int m = 0; m < NV; m++) {
      const int c = x * V + m * STEP;
      if (c < a.n) {
        if constexpr (MODE == NORM_Y) stv<T, V>((T *)a.y + row * a.ly + c, s[m]);
        else store_q<V>(a.q + row * a.lq + c, s[m], scale);
      }
    }
  } else {
    float ss = 0.f, top = 0.f;
    for (int c = x * V; c < a.n; c += STEP) {
      const VecOf<T, V> v = ldv<T, V>(xp + c, true);
      VecOf<T, V> r;
      if (MODE != NORM_QUANT && rp) r = ldv<T, V>(rp + c, true);
      float s[V];
#pragma unroll
      for (int i = 0; i < V; i++) {
        s[i] = v.f(i);
        if (MODE != NORM_QUANT && rp) s[i] = to_storage<T>(s[i] + r.f(i));
        if (MODE == NORM_QUANT) top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(fabsf(s[i]))));
        else ss = fmaf(s[i], s[i], ss);
      }
      if (MODE != NORM_QUANT && sp) stv<T, V>(sp + c, s);
    }
    float rstd = 1.f;
    if constexpr (MODE != NORM_QUANT) {
      ss = row_sum<TPR>(ss, sh[0]);
      rstd = 1.f / sqrtf(ss / (float)a.n + a.eps);
    }
    // the sum where it was kept (it may have replaced x or r), else made again
    auto value = [&](int c, float *y) {
      const VecOf<T, V> v = ldv<T, V>(MODE != NORM_QUANT && sp ? sp + c : xp + c, true);
      VecOf<T, V> r, w;
      const bool add = MODE != NORM_QUANT && rp && !sp;
      if (add) r = ldv<T, V>(rp + c, true);
      if (MODE != NORM_QUANT && wp) w = ldv<T, V>(wp + c, true);
#pragma unroll
      for (int i = 0; i < V; i++) {
        float s = v.f(i);
        if (add) s = to_storage<T>(s + r.f(i));
        y[i] = MODE == NORM_QUANT ? s : s * rstd * (wp ? w.f(i) : 1.f);
      }
    };
    float scale = 0.f;
    if constexpr (MODE != NORM_Y) {
      if constexpr (MODE == NORM_Q)
        for (int c = x * V; c < a.n; c += STEP) {
          float y[V];
          value(c, y);
#pragma unroll
          for (int i = 0; i < V; i++) top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(fabsf(y[i]))));
        }
      scale = row_max<TPR>(top, sh[1]) * (1.f / 127.f);
      if (x == 0) a.scale[row] = scale;
    }
    for (int c = x * V; c < a.n; c += STEP) {
      float y[V];
      value(c, y);
      if constexpr (MODE == NORM_Y) stv<T, V>((T *)a.y + row * a.ly + c, y);
      else store_q<V>(a.q + row * a.lq + c, y, scale);
    }
  }
}

// dx = rstd (w dy - s rstd^2 sum(w dy s) / n) + ds; dw = sum over rows of
// dy s rstd.  Blocks walk rows with a stride of the grid and keep dw of their
// columns in registers; NV = 0: long rows, dw comes from k_norm_dw.
template <typename T, int V, int TPR, int NV>
__global__ __launch_bounds__(256) void k_norm_adj(NormArgs a) {
  constexpr int RPB = 256 / TPR, STEP = TPR * V;
  __shared__ float sh[2][2][4];
  const int x = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const T *wp = (const T *)a.w;
  if constexpr (NV > 0) {
    float dw[NV][V], w[NV][V];
#pragma unroll
    for (int m = 0; m < NV; m++) {
      const int c = x * V + m * STEP;
      const VecOf<T, V> v = ldv<T, V>(wp + c, wp && c < a.n);
#pragma unroll
      for (int i = 0; i < V; i++) {
        dw[m][i] = 0.f;
        w[m][i] = wp ? v.f(i) : 1.f;
      }
    }
    int par = 0;
    for (long long row = (long long)blockIdx.x * RPB + sub; row < a.rows; row += (long long)gridDim.x * RPB) {
      VecOf<T, V> s[NV], g[NV], e[NV];
#pragma unroll
      for (int m = 0; m < NV; m++) {
        const int c = x * V + m * STEP;
        s[m] = ldv<T, V>((const T *)a.s + row * a.ls + c, c < a.n);
        g[m] = ldv<T, V>((const T *)a.dy + row * a.ldy + c, c < a.n);
        if (a.ds) e[m] = ldv<T, V>((const T *)a.ds + row * a.lds + c, c < a.n);
      }
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int m = 0; m < NV; m++)
#pragma unroll
        for (int i = 0; i < V; i++) {
          const float v = s[m].f(i);
          ss = fmaf(v, v, ss);
          dot = fmaf(w[m][i] * g[m].f(i), v, dot);
        }
      ss = wave_total(ss);
      dot = wave_total(dot);
      if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) {
          sh[par][0][threadIdx.x >> 6] = ss;
          sh[par][1][threadIdx.x >> 6] = dot;
        }
        __syncthreads();
        ss = (sh[par][0][0] + sh[par][0][1]) + (sh[par][0][2] + sh[par][0][3]);
        dot = (sh[par][1][0] + sh[par][1][1]) + (sh[par][1][2] + sh[par][1][3]);
        par ^= 1;  // the next row's sums go to the other half
      }
      const float rstd = 1.f / sqrtf(ss / (float)a.n + a.eps), k = dot * rstd * rstd / (float)a.n;
#pragma unroll
      for (int m = 0; m < NV; m++) {
        const int c = x * V + m * STEP;
        float o[V];
#pragma unroll
        for (int i = 0; i < V; i++) {
          const float v = s[m].f(i), gy = g[m].f(i);
          o[i] = rstd * fmaf(-v, k, w[m][i] * gy) + (a.ds ? e[m].f(i) : 0.f);
          dw[m][i] = fmaf(gy, v * rstd, dw[m][i]);
        }
        if (a.dx && c < a.n) stv<T, V>((T *)a.dx + row * a.ldx + c, o);
      }
    }
    if (!a.part) return;
    float *pp = a.part + (long long)blockIdx.x * a.n;
    if constexpr (RPB == 1) {
#pragma unroll
      for (int m = 0; m < NV; m++)
#pragma unroll
        for (int i = 0; i < V; i++)
          if (x * V + m * STEP + i < a.n) pp[x * V + m * STEP + i] = dw[m][i];
    } else {  // join the block's rows
      __shared__ float red[RPB][NV * V * TPR];
#pragma unroll
      for (int m = 0; m < NV; m++)
#pragma unroll
        for (int i = 0; i < V; i++) red[sub][x * V + m * STEP + i] = dw[m][i];
      __syncthreads();
      for (int c = threadIdx.x; c < a.n; c += 256) {
        float v = red[0][c];
#pragma unroll
        for (int m = 1; m < RPB; m++) v += red[m][c];
        pp[c] = v;
      }
    }
  } else {
    const long long row = flat_block();
    if (row >= a.rows) return;
    const T *sp = (const T *)a.s + row * a.ls, *gp = (const T *)a.dy + row * a.ldy;
    float ss = 0.f, dot = 0.f;
    for (int c = x; c < a.n; c += 256) {
      const float v = ldf(sp, c);
      ss = fmaf(v, v, ss);
      dot = fmaf((wp ? ldf(wp, c) : 1.f) * ldf(gp, c), v, dot);
    }
    ss = row_sum<256>(ss, sh[0][0]);
    dot = row_sum<256>(dot, sh[0][1]);
    const float rstd = 1.f / sqrtf(ss / (float)a.n + a.eps), k = dot * rstd * rstd / (float)a.n;
    if (x == 0 && a.rstd) a.rstd[row] = rstd;
    if (a.dx)
      for (int c = x; c < a.n; c += 256) {
        const float e = a.ds ? ldf((const T *)a.ds + row * a.lds, c) : 0.f;
        stf((T *)a.dx + row * a.ldx, c, rstd * fmaf(-ldf(sp, c), k, (wp ? ldf(wp, c) : 1.f) * ldf(gp, c)) + e);
      }
  }
}

// dw of long rows: a block sums one slice of the rows for 256 columns
template <typename T>
__global__ void k_norm_dw(NormArgs a, int slices) {
  const int c = (int)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.n) return;
  const long long per = (a.rows + slices - 1) / slices, r0 = blockIdx.y * per;
  const long long r1 = r0 + per < a.rows ? r0 + per : a.rows;
  float v = 0.f;
  for (long long r = r0; r < r1; r++)
    v = fmaf(ldf((const T *)a.dy + r * a.ldy, c), ldf((const T *)a.s + r * a.ls, c) * a.rstd[r], v);
  a.part[(long long)blockIdx.y * a.n + c] = v;
}

// Threads per row and vectors per thread for rows of n in vectors of V:
// a wavefront up to 4 vectors a lane, then a block up to 8 (scalar access:
// up to 32 elements), else 0 (the row is read again for each pass).
struct NormGeom {
  int tpr, nv;
};
static NormGeom norm_geom(int n, int V) {
  const int q = (n + V - 1) / V;
  if (V == 1) {
    if (q <= 64 * 4) return {64, 4};
    if (q <= 256 * 8) return {256, 8};
    if (q <= 256 * 32) return {256, 32};
    return {256, 0};
  }
  if (q <= 64) return {64, 1};
  if (q <= 128) return {64, 2};
  if (q <= 256) return {64, 4};
  if (q <= 512) return {256, 2};
  if (q <= 1024) return {256, 4};
  if (q <= 2048) return {256, 8};
  return {256, 0};
}
// Blocks of the adjoint: a few rows each, so that their dw partials are few
static int norm_adj_blocks(long long rows, int rpb) {
  const long long b = (rows + rpb - 1) / rpb;
  return (int)(b < 1024 ? b : 1024);
}

template <typename T, int V, int TPR, int NV>
hipError_t norm_go(const NormArgs &a, int mode, hipStream_t s) {
  constexpr int RPB = 256 / TPR;
  const dim3 grid = flat_grid((a.rows + RPB - 1) / RPB);
  if (mode == NORM_Y) k_norm<T, V, TPR, NV, NORM_Y><<<grid, 256, 0, s>>>(a);
  else if (mode == NORM_Q) k_norm<T, V, TPR, NV, NORM_Q><<<grid, 256, 0, s>>>(a);
  else if (mode == NORM_QUANT) k_norm<T, V, TPR, NV, NORM_QUANT><<<grid, 256, 0, s>>>(a);
  else k_norm_adj<T, V, TPR, NV><<<NV > 0 ? dim3(norm_adj_blocks(a.rows, RPB)) : grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

constexpr int NORM_ADJ = 3;
template <typename T, int V>
hipError_t norm_vec(const NormArgs &a, int mode, hipStream_t s) {
  const NormGeom g = norm_geom(a.n, V);
  if constexpr (V == 1) {
    if (g.tpr == 64) return norm_go<T, 1, 64, 4>(a, mode, s);
    if (g.nv == 8) return norm_go<T, 1, 256, 8>(a, mode, s);
    if (g.nv == 32) return norm_go<T, 1, 256, 32>(a, mode, s);
    return norm_go<T, 1, 256, 0>(a, mode, s);
  } else {
    if (g.tpr == 64) {
      if (g.nv == 1) return norm_go<T, V, 64, 1>(a, mode, s);
      if (g.nv == 2) return norm_go<T, V, 64, 2>(a, mode, s);
      return norm_go<T, V, 64, 4>(a, mode, s);
    }
    if (g.nv == 2) return norm_go<T, V, 256, 2>(a, mode, s);
    if (g.nv == 4) return norm_go<T, V, 256, 4>(a, mode, s);
    if (g.nv == 8) return norm_go<T, V, 256, 8>(a, mode, s);
    return norm_go<T, 1, 256, 0>(a, mode, s);
  }
}
static hipError_t norm_dispatch(int dtype, bool vec, const NormArgs &a, int mode, hipStream_t s) {
  if (dtype == PR_BF16) return vec ? norm_vec<uint16_t, 8>(a, mode, s) : norm_vec<uint16_t, 1>(a, mode, s);
  return vec ? norm_vec<float, 4>(a, mode, s) : norm_vec<float, 1>(a, mode, s);
}

}  // namespace pr

using namespace pr;

namespace {

#define HIPCHK(expr)                                                                        \
  do {                                                                                      \
    hipError_t e_ = (expr);                                                                 \
    if (e_ != hipSuccess) return fail(PR_EHIP, "%s: %s", #expr, hipGetErrorString(e_));     \
  } while (0)

constexpr int DW_SLICES = 64;

int norm_check(const pr_norm_problem *p) {
  if (!p) return fail(PR_EINVAL, "problem is NULL");
  if (p->dtype != PR_F32 && p->dtype != PR_BF16) return fail(PR_EINVAL, "unknown dtype %d", p->dtype);
  if (p->rows < 1 || p->n < 1) return fail(PR_EINVAL, "sizes must be >= 1 (rows=%lld n=%d)", p->rows, p->n);
  if (!(p->eps >= 0.f) || p->eps > 3.0e38f) return fail(PR_EINVAL, "eps must be >= 0 and finite");
  if (p->rows > 2147483647LL || p->n > (1 << 30)) return fail(PR_EUNSUPPORTED, "problem too large");
  return PR_OK;
}

bool has(const pr_rows *r) { return r && r->p; }
bool vec_ok(const pr_rows *r, int V, int bytes) {
  return !has(r) || (((uintptr_t)r->p % bytes) == 0 && r->ld % V == 0);
}

int norm_run(const pr_norm_problem *p, const pr_rows *x, const pr_rows *r, const void *w, const pr_rows *s,
             const pr_rows *y, const pr_rows *q, float *scale, int mode, void *stream) {
  NormArgs a{};
  a.x = x->p; a.lx = x->ld;
  if (has(r)) { a.r = r->p; a.lr = r->ld; }
  if (has(s)) { a.s = s->p; a.ls = s->ld; }
  if (has(y)) { a.y = y->p; a.ly = y->ld; }
  if (has(q)) { a.q = (int8_t *)q->p; a.lq = q->ld; }
  a.w = w; a.scale = scale; a.rows = p->rows; a.n = p->n; a.eps = p->eps;
  const int V = p->dtype == PR_BF16 ? 8 : 4;
  const bool vec = p->n % V == 0 && vec_ok(x, V, 16) && vec_ok(r, V, 16) && vec_ok(s, V, 16) && vec_ok(y, V, 16) &&
                   vec_ok(q, V, V) && ((uintptr_t)w & 15) == 0;
  HIPCHK(norm_dispatch(p->dtype, vec, a, mode, (hipStream_t)stream));
  return PR_OK;
}

}  // namespace

extern "C" {

int pararnn_rmsnorm(const pr_norm_problem *p, const pr_rows *x, const pr_rows *r, const void *w, const pr_rows *sum_out,
                    const pr_rows *y, const pr_rows *q, float *scale, void *stream) {
  clear_error();
  const int rc = norm_check(p);
  if (rc != PR_OK) return rc;
  if (!has(x)) return fail(PR_EINVAL, "x is required");
  if (has(y) == has(q)) return fail(PR_EINVAL, "exactly one of y and q is required");
  if (has(q) && !scale) return fail(PR_EINVAL, "scale is required with q");
  return norm_run(p, x, r, w, sum_out, y, q, scale, has(q) ? NORM_Q : NORM_Y, stream);
}

int pararnn_quant_rows(const pr_norm_problem *p, const pr_rows *x, const pr_rows *q, float *scale, void *stream) {
  clear_error();
  const int rc = norm_check(p);
  if (rc != PR_OK) return rc;
  if (!has(x) || !has(q) || !scale) return fail(PR_EINVAL, "x, q and scale are required");
  return norm_run(p, x, nullptr, nullptr, nullptr, nullptr, q, scale, NORM_QUANT, stream);
}

size_t pararnn_rmsnorm_workspace_bytes(const pr_norm_problem *p) {
  clear_error();
  if (norm_check(p) != PR_OK) return 0;
  size_t most = 0;
  for (int V : {1, p->dtype == PR_BF16 ? 8 : 4}) {
    const NormGeom g = norm_geom(p->n, V);
    const size_t blocks = g.nv ? (size_t)norm_adj_blocks(p->rows, 256 / g.tpr) : (size_t)DW_SLICES;
    const size_t need = blocks * p->n * 4 + (g.nv ? 0 : (size_t)p->rows * 4 + 256);
    most = need > most ? need : most;
  }
  return (most + 255) & ~(size_t)255;
}

int pararnn_rmsnorm_adjoint(const pr_norm_problem *p, const pr_rows *s, const void *w, const pr_rows *dy,
                            const pr_rows *dsum, const pr_rows *dx, float *dw, void *workspace, size_t ws_bytes,
                            void *stream) {
  clear_error();
  const int rc = norm_check(p);
  if (rc != PR_OK) return rc;
  if (!has(s) || !has(dy)) return fail(PR_EINVAL, "s and dy are required");
  const size_t need = pararnn_rmsnorm_workspace_bytes(p);
  if (!workspace || ws_bytes < need) return fail(PR_EWORKSPACE, "workspace %zu bytes < %zu", ws_bytes, need);
  if (((uintptr_t)workspace & 255) != 0) return fail(PR_EINVAL, "workspace must be 256-byte aligned");
  NormArgs a{};
  a.s = s->p; a.ls = s->ld; a.dy = dy->p; a.ldy = dy->ld;
  if (has(dsum)) { a.ds = dsum->p; a.lds = dsum->ld; }
  if (has(dx)) { a.dx = dx->p; a.ldx = dx->ld; }
  a.w = w; a.rows = p->rows; a.n = p->n; a.eps = p->eps;
  const int V0 = p->dtype == PR_BF16 ? 8 : 4;
  const bool vec = p->n % V0 == 0 && vec_ok(s, V0, 16) && vec_ok(dy, V0, 16) && vec_ok(dsum, V0, 16) &&
                   vec_ok(dx, V0, 16) && ((uintptr_t)w & 15) == 0;
  const NormGeom g = norm_geom(p->n, vec ? V0 : 1);
  a.part = dw ? (float *)workspace : nullptr;
  if (!g.nv && dw) a.rstd = (float *)((char *)workspace + (((size_t)DW_SLICES * p->n * 4 + 255) & ~(size_t)255));
  hipStream_t st = (hipStream_t)stream;
  HIPCHK(norm_dispatch(p->dtype, vec, a, NORM_ADJ, st));
  if (!dw) return PR_OK;
  int parts = norm_adj_blocks(p->rows, 256 / g.tpr);
  if (!g.nv) {
    parts = DW_SLICES;
    const dim3 grid((unsigned)((p->n + 255) / 256), DW_SLICES);
    if (p->dtype == PR_BF16) k_norm_dw<uint16_t><<<grid, 256, 0, st>>>(a, DW_SLICES);
    else k_norm_dw<float><<<grid, 256, 0, st>>>(a, DW_SLICES);
    HIPCHK(hipGetLastError());
  }
  HIPCHK(launch_part_sum(a.part, parts, p->n, p->n, dw, st));
  return PR_OK;
}

}  // extern "C"
