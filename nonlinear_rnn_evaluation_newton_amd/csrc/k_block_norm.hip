// Norms around a block, joined with its gate and the residual's scale:
//   u = x rstd(x) w scale act(z),  t = residual + u,  y = t rstd(t) w_next
// and the adjoint, from the stored t (x^ = x rstd1, t^ = t rstd2):
//   gt = dt + rstd2 (w_next dy - t^ mean(w_next dy t^)),  dresidual = gt
//   e = gt w scale act(z),  dx = rstd1 (e - x^ mean(e x^)),
//   dz = gt w scale x^ act'(z),  q = sum over rows of gt act(z) x^,
//   dw = scale q,  dscale = w q,  dw_next = sum over rows of dy t^
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
  float eps;
};

// act(z) and its derivative
struct Act {
  float v, d;
};
__device__ inline Act bn_act(int gate, float z) {
  const float p = fsigm(z);
  if (gate == PR_GATE_SIGMOID) return Act{p, p * (1.f - p)};
  return Act{z * p, p * fmaf(z, 1.f - p, 1.f)};
}
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

// Long rows: a block reads its row again for each pass.
template <typename T>
__global__ __launch_bounds__(256) void k_bn_long(BnArgs a) {
  __shared__ float sh[2][4];
  const long long row = flat_block();
  if (row >= a.rows) return;
  const T *xp = (const T *)a.x + row * a.lx, *zp = (const T *)a.z + row * a.lz, *rp = (const T *)a.res + row * a.lres;
  T *tp = (T *)a.t + row * a.lt;
  float ss = 0.f;
  for (int c = threadIdx.x; c < a.n; c += 256) {
    const float v = ldf(xp, c);
    ss = fmaf(v, v, ss);
  }
  const float rstd = 1.f / sqrtf(block_sum(ss, sh[0]) / (float)a.n + a.eps);
  ss = 0.f;
  for (int c = threadIdx.x; c < a.n; c += 256) {
    float u = ldf(xp, c) * rstd * (at1<T>(a.w, c) * at1<T>(a.scale, c));
    if (a.z) u *= bn_act(a.gate, ldf(zp, c)).v;
    const float t = to_storage<T>(a.res ? ldf(rp, c) + u : u);
    stf(tp, c, t);
    ss = fmaf(t, t, ss);
  }
  if (!a.y) return;
  const float rstd2 = 1.f / sqrtf(block_sum(ss, sh[1]) / (float)a.n + a.eps);
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
  float ss = 0.f, st = 0.f, dot = 0.f;
  for (int c = threadIdx.x; c < a.n; c += 256) {
    const float v = ldf((const T *)a.x + row * a.lx, c);
    ss = fmaf(v, v, ss);
    if (a.dy) {
      const float t = ldf((const T *)a.t + row * a.lt, c);
      st = fmaf(t, t, st);
      dot = fmaf(at1<T>(a.wn, c) * ldf((const T *)a.dy + row * a.ldy, c), t, dot);
    }
  }
  ss = block_sum(ss, sh[0]);
  st = block_sum(st, sh[1]);
  dot = block_sum(dot, sh[2]);
  if (threadIdx.x == 0) {
    float *o = a.stat + row * 3;
    const float n = (float)a.n, rstd2 = 1.f / sqrtf(st / n + a.eps);
    o[0] = 1.f / sqrtf(ss / n + a.eps);
    o[1] = rstd2;
    o[2] = dot / n * rstd2 * rstd2;
  }
}
// q and dw_next: a block sums one slice of the rows for 256 columns
template <typename T>
__global__ __launch_bounds__(256) void k_bn_adj_cols(BnArgs a, int slices) {
  const int c = (int)blockIdx.x * 256 + threadIdx.x;
  if (c >= a.n) return;
  const long long per = (a.rows + slices - 1) / slices, r0 = blockIdx.y * per;
  const long long r1 = r0 + per < a.rows ? r0 + per : a.rows;
  float q = 0.f, wn = 0.f;
  for (long long r = r0; r < r1; r++) {
    const BnRow s{a.stat[r * 3], a.stat[r * 3 + 1], a.stat[r * 3 + 2]};
    const float xh = ldf((const T *)a.x + r * a.lx, c) * s.rstd1;
    const float act = a.z ? bn_act(a.gate, ldf((const T *)a.z + r * a.lz, c)).v : 1.f;
    q = fmaf(bn_gt<T>(a, s, r, c) * act, xh, q);
    if (a.dy)
      wn = fmaf(ldf((const T *)a.dy + r * a.ldy, c), ldf((const T *)a.t + r * a.lt, c) * s.rstd2, wn);
  }
  a.part[(blockIdx.y * 2LL) * a.n + c] = q;
  a.part[(blockIdx.y * 2LL + 1) * a.n + c] = wn;
}
template <typename T>
__global__ __launch_bounds__(256) void k_bn_adj_long(BnArgs a) {
  __shared__ float sh[4];
  const long long row = flat_block();
  if (row >= a.rows) return;
  const BnRow s{a.stat[row * 3], a.stat[row * 3 + 1], a.stat[row * 3 + 2]};
  const T *xp = (const T *)a.x + row * a.lx, *zp = (const T *)a.z + row * a.lz;
  float dot = 0.f;
  for (int c = threadIdx.x; c < a.n; c += 256) {
    float e = bn_gt<T>(a, s, row, c) * (at1<T>(a.w, c) * at1<T>(a.scale, c));
    if (a.z) e *= bn_act(a.gate, ldf(zp, c)).v;
    dot = fmaf(e, ldf(xp, c), dot);
  }
  const float k1 = block_sum(dot, sh) / (float)a.n * s.rstd1 * s.rstd1;
  for (int c = threadIdx.x; c < a.n; c += 256) {
    const float gt = bn_gt<T>(a, s, row, c), ws = at1<T>(a.w, c) * at1<T>(a.scale, c), x = ldf(xp, c);
    const Act act = a.z ? bn_act(a.gate, ldf(zp, c)) : Act{1.f, 0.f};
    if (a.dres) stf((T *)a.dres + row * a.ldres, c, gt);
    if (a.dz) stf((T *)a.dz + row * a.ldz, c, gt * ws * (x * s.rstd1) * act.d);
    if (a.dx) stf((T *)a.dx + row * a.ldx, c, s.rstd1 * fmaf(-x, k1, gt * ws * act.v));
  }
}

// The weights' gradients from the sums of the columns: q [n] becomes dw and dscale.
template <typename T>
__global__ __launch_bounds__(256) void k_bn_weights(const float *q, const void *w, const void *scale, int n, float *dw,
                                                    float *dscale) {
  const int c = (int)blockIdx.x * 256 + threadIdx.x;
  if (c >= n) return;
  const float v = q[c];
  if (dw) dw[c] = v * at1<T>(scale, c);
  if (dscale) dscale[c] = v * at1<T>(w, c);
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
  a->rows = p->rows; a->n = p->n; a->gate = p->gate; a->eps = p->eps;
  return PR_OK;
}

struct BnPlan {
  size_t off_part, off_q, bytes;
  int parts;
};
BnPlan bn_plan(const pr_block_norm_problem *p) {
  BnPlan pl;
  pl.parts = BN_SLICES;
  size_t o = align256((size_t)p->rows * 12);
  pl.off_part = o; o = align256(o + (size_t)pl.parts * 2 * p->n * 4);
  pl.off_q = o; o = align256(o + (size_t)p->n * 4);
  pl.bytes = o;
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
  a.stat = (float *)ws;
  a.part = (float *)(ws + pl.off_part);
  float *q = (float *)(ws + pl.off_q);
  hipStream_t s = (hipStream_t)stream;
  const dim3 grid = flat_grid(p->rows), cols((unsigned)((p->n + 255) / 256), (unsigned)pl.parts);
  const bool bf = p->dtype == PR_BF16, sums = gr->w || gr->scale || gr->w_next;
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
  if (gr->w || gr->scale) {
    HIPCHK(launch_part_sum(a.part, pl.parts, 2LL * p->n, p->n, q, s));
    const unsigned nb = (unsigned)((p->n + 255) / 256);
    if (bf) k_bn_weights<uint16_t><<<nb, 256, 0, s>>>(q, w, scale, p->n, gr->w, gr->scale);
    else k_bn_weights<float><<<nb, 256, 0, s>>>(q, w, scale, p->n, gr->w, gr->scale);
    HIPCHK(hipGetLastError());
  }
  if (gr->w_next) HIPCHK(launch_part_sum(a.part + p->n, pl.parts, 2LL * p->n, p->n, gr->w_next, s));
  return PR_OK;
}

}  // extern "C"
