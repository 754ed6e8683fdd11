// Weights in 4 bits with a scale and a zero point for each group of columns:
// their product with few rows, the 4-bit form of a matrix, and the values that
// it stands for.
#include "pararnn.h"
#include "ssm.h"
#include "vec.h"

namespace pr {

struct W4Args {
  const void *x, *scale, *zero, *bias;  // zero, bias may be null
  const uint8_t *q;
  void *out;
  long long ldx, ldq, ldo;
  int M, N, K, group, G;  // G: groups of a row
};

// One wavefront for each row of weights and eight rows of x.
template <typename T>
__global__ __launch_bounds__(256) void k_w4_plain(W4Args a) {
  const int n = (int)blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63, m0 = (int)blockIdx.y * 8;
  if (n >= a.N) return;
  const uint8_t *qp = a.q + n * a.ldq;
  float acc[8] = {};
  for (int k = lane; k < a.K; k += 64) {
    const int g = k / a.group;
    const float s = ldf((const T *)a.scale, (long long)n * a.G + g);
    const float z = a.zero ? ldf((const T *)a.zero, (long long)n * a.G + g) : 8.f;
    const float w = ((float)((qp[k >> 1] >> (4 * (k & 1))) & 15) - z) * s;
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (m0 + i < a.M) acc[i] = fmaf(w, ldf((const T *)a.x + (m0 + i) * a.ldx, k), acc[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float v = wave_total(acc[i]);
    if (lane == 0 && m0 + i < a.M)
      stf((T *)a.out + (m0 + i) * a.ldo, n, v + (a.bias ? ldf((const T *)a.bias, n) : 0.f));
  }
}

struct W4QuantArgs {
  void *w, *scale, *zero;  // zero may be null
  uint8_t *q;
  long long ldw, ldq;
  int N, K, group, G;
};

// y / s to the nearest, ties to even; s > 0 and finite
__device__ inline float w4_round(float y, float s) { return rintf(__fdiv_rn(y, s)); }

// L lanes (a power of two) for each group, eight columns each at a time.
template <typename T, int L>
__global__ __launch_bounds__(256) void k_w4_quant(W4QuantArgs a) {
  const long long id = flat_block() * (256 / L) + threadIdx.x / L;  // row and group
  const int lane = threadIdx.x % L;
  const bool on = id < (long long)a.N * a.G;
  const int g = on ? (int)(id % a.G) : 0;
  const long long n = on ? id / a.G : 0;
  const int k0 = g * a.group, k1 = on ? (a.K - k0 < a.group ? a.K : k0 + a.group) : k0;
  const T *wp = (const T *)a.w + n * a.ldw;
  // the largest of max(w, 0) and of max(-w, 0), compared by their bits: a NaN wins
  unsigned hi = 0, lo = 0;
  for (int k = k0 + lane * 8; k < k1; k += L * 8) {
    const VecU<T, 8> v = ldu<T, 8>(wp + k, k1 - k);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float f = v.f(i);
      const unsigned bits = __float_as_uint(fabsf(f));
      if (f > 0.f || f != f) hi = max(hi, bits);
      else lo = max(lo, bits);
    }
  }
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) {
    hi = max(hi, (unsigned)__shfl_xor((int)hi, o, 64));
    lo = max(lo, (unsigned)__shfl_xor((int)lo, o, 64));
  }
  const float fh = __uint_as_float(hi), fl = __uint_as_float(lo);
  T st;
  stf(&st, 0, a.zero ? (fh + fl) * (1.f / 15.f) : __uint_as_float(max(hi, lo)) * (1.f / 7.f));
  const float s = ldf(&st, 0);
  const bool plain = s > 0.f && s < __builtin_inff();
  float z = 8.f;
  if (a.zero) z = plain ? fminf(fmaxf(w4_round(fl, s), 0.f), 15.f) : s == 0.f ? 0.f : 8.f;
  if (on && lane == 0) {
    ((T *)a.scale)[id] = st;
    if (a.zero) stf((T *)a.zero, id, z);
  }
  for (int k = k0 + lane * 8; k < k1; k += L * 8) {
    const int c = k1 - k;
    const VecU<T, 8> v = ldu<T, 8>(wp + k, c);
    unsigned word = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float f = plain ? w4_round(v.f(i), s) + z : z;
      word |= (unsigned)(int)fminf(fmaxf(f, 0.f), 15.f) << (4 * i);
    }
    uint8_t *qp = a.q + n * a.ldq + (k >> 1);
    if (c >= 8) {
      reinterpret_cast<Packed<uint8_t, 4> *>(qp)->v = word;
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (2 * i < c) qp[i] = (uint8_t)(word >> (8 * i));
    }
  }
}

// Eight columns a thread.
template <typename T>
__global__ __launch_bounds__(256) void k_w4_dequant(W4QuantArgs a, int per) {
  const long long id = flat_block() * 256 + threadIdx.x;
  const long long n = id / per;
  const int k = (int)(id % per) * 8, c = a.K - k;
  if (n >= a.N) return;
  const uint8_t *qp = a.q + n * a.ldq + (k >> 1);
  unsigned word = 0;
  if (c >= 8) {
    word = reinterpret_cast<const Packed<uint8_t, 4> *>(qp)->v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (2 * i < c) word |= (unsigned)qp[i] << (8 * i);
  }
  const long long g = n * a.G + k / a.group;  // (groups are multiples of 32)
  const float s = ldf((const T *)a.scale, g), z = a.zero ? ldf((const T *)a.zero, g) : 8.f;
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; i++) o[i] = ((float)((word >> (4 * i)) & 15) - z) * s;
  stu<T, 8>((T *)a.w + n * a.ldw + k, o, c);
}

template <typename T>
hipError_t w4_quant_go(const W4QuantArgs &a, hipStream_t s) {
  const long long groups = (long long)a.N * a.G;
#define PR_Q(L)                                                                    \
  {                                                                                \
    k_w4_quant<T, L><<<flat_grid((groups * L + 255) / 256), 256, 0, s>>>(a);       \
    return hipGetLastError();                                                      \
  }
  if (a.group <= 32) PR_Q(4)
  if (a.group <= 64) PR_Q(8)
  if (a.group <= 128) PR_Q(16)
  if (a.group <= 256) PR_Q(32)
  PR_Q(64)
#undef PR_Q
}

}  // namespace pr

using namespace pr;

namespace {

#define HIPCHK(expr)                                                                        \
  do {                                                                                      \
    hipError_t e_ = (expr);                                                                 \
    if (e_ != hipSuccess) return fail(PR_EHIP, "%s: %s", #expr, hipGetErrorString(e_));     \
  } while (0)

constexpr int W4_MAX = 1 << 24;

int w4_check(int dtype, int M, int N, int K, int group) {
  if (dtype != PR_F32 && dtype != PR_BF16) return fail(PR_EINVAL, "unknown dtype %d", dtype);
  if (M < 1 || N < 1 || K < 1) return fail(PR_EINVAL, "sizes must be >= 1 (M=%d N=%d K=%d)", M, N, K);
  if (group < 1) return fail(PR_EINVAL, "group = %d", group);
  if (group % 32 != 0) return fail(PR_EUNSUPPORTED, "group = %d: a multiple of 32", group);
  if (M > (1 << 21) || N > W4_MAX || K > W4_MAX)
    return fail(PR_EUNSUPPORTED, "M = %d, N = %d, K = %d: at most 2^21, 2^24, 2^24", M, N, K);
  return PR_OK;
}

int w4_groups(int K, int group) { return (int)(((long long)K + group - 1) / group); }

}  // namespace

extern "C" {

int pararnn_gemm_w4(int dtype, int M, int N, int K, int group, const void *x, long long ldx, const unsigned char *q,
                    long long ldq, const void *scale, const void *zero, const void *bias, void *out, long long ldo,
                    void *stream) {
  clear_error();
  const int rc = w4_check(dtype, M, N, K, group);
  if (rc != PR_OK) return rc;
  if (!x || !q || !scale || !out) return fail(PR_EINVAL, "x, q, scale and out are required");
  // one row has no stride: whatever stands for it is not looked at
  if (M == 1) { ldx = K; ldo = N; }
  if (N == 1) ldq = (K + 1) / 2;
  if (ldx < K || ldq < (K + 1) / 2 || ldo < N)
    return fail(PR_EINVAL, "row strides %lld, %lld, %lld are below K = %d, (K + 1) / 2, N = %d", ldx, ldq, ldo, K, N);
  W4Args a{};
  a.x = x; a.q = q; a.scale = scale; a.zero = zero; a.bias = bias; a.out = out;
  a.ldx = ldx; a.ldq = ldq; a.ldo = ldo; a.M = M; a.N = N; a.K = K; a.group = group; a.G = w4_groups(K, group);
  const dim3 grid((unsigned)((N + 3) / 4), (unsigned)((M + 7) / 8));
  if ((double)grid.x * grid.y * 256 >= 4294967296.0) return fail(PR_EUNSUPPORTED, "problem too large: %d x %d results", M, N);
  if (grid.y > 65535) return fail(PR_EUNSUPPORTED, "M = %d", M);
  if (dtype == PR_BF16) k_w4_plain<uint16_t><<<grid, 256, 0, (hipStream_t)stream>>>(a);
  else k_w4_plain<float><<<grid, 256, 0, (hipStream_t)stream>>>(a);
  HIPCHK(hipGetLastError());
  return PR_OK;
}

int pararnn_quant_w4(int dtype, int N, int K, int group, const void *w, long long ldw, unsigned char *q, long long ldq,
                     void *scale, void *zero, void *stream) {
  clear_error();
  const int rc = w4_check(dtype, 1, N, K, group);
  if (rc != PR_OK) return rc;
  if (!w || !q || !scale) return fail(PR_EINVAL, "w, q and scale are required");
  if (N == 1) { ldw = K; ldq = (K + 1) / 2; }
  if (ldq < (K + 1) / 2) return fail(PR_EINVAL, "row stride %lld is below (K + 1) / 2 = %d", ldq, (K + 1) / 2);
  W4QuantArgs a{(void *)w, scale, zero, q, ldw, ldq, N, K, group, w4_groups(K, group)};
  HIPCHK(dtype == PR_BF16 ? w4_quant_go<uint16_t>(a, (hipStream_t)stream) : w4_quant_go<float>(a, (hipStream_t)stream));
  return PR_OK;
}

int pararnn_dequant_w4(int dtype, int N, int K, int group, const unsigned char *q, long long ldq, const void *scale,
                       const void *zero, void *w, long long ldw, void *stream) {
  clear_error();
  const int rc = w4_check(dtype, 1, N, K, group);
  if (rc != PR_OK) return rc;
  if (!w || !q || !scale) return fail(PR_EINVAL, "q, scale and w are required");
  if (N == 1) { ldw = K; ldq = (K + 1) / 2; }
  if (ldw < K || ldq < (K + 1) / 2)
    return fail(PR_EINVAL, "row strides %lld, %lld are below K = %d, (K + 1) / 2", ldw, ldq, K);
  W4QuantArgs a{w, (void *)scale, (void *)zero, (uint8_t *)q, ldw, ldq, N, K, group, w4_groups(K, group)};
  const int per = (K + 7) / 8;
  const dim3 grid = flat_grid(((long long)N * per + 255) / 256);
  if (dtype == PR_BF16) k_w4_dequant<uint16_t><<<grid, 256, 0, (hipStream_t)stream>>>(a, per);
  else k_w4_dequant<float><<<grid, 256, 0, (hipStream_t)stream>>>(a, per);
  HIPCHK(hipGetLastError());
  return PR_OK;
}

}  // extern "C"
