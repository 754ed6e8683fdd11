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
  float rgroup;           // 32 / group
  int slice;              // columns of a wavefront
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4v __attribute__((ext_vector_type(4)));
constexpr int W4_CH = 128;  // columns of a wavefront's step: 16 bytes of 4-bit numbers a lane

// Weights are multiplied as sixteenths, exact powers of two away from their values: up
// to 128 columns are summed before their scale comes in, and of rows below 1e36 such a
// sum, of at most two for each, stays below fp32's largest.  The result is multiplied by 16.
constexpr float W4_UNIT = 16.f;

// Operands of v_mfma_f32_16x16x32_bf16 for 8 adjacent columns k0..k7 of a lane, in
// the order k0 k4, k1 k5, k2 k6, k3 k7: both operands have the same, and a product's
// terms may come in any.
__device__ inline bf16x8 words(unsigned a, unsigned b, unsigned c, unsigned d) {
  return __builtin_bit_cast(bf16x8, u32x4v{a, b, c, d});
}
__device__ inline unsigned halves(unsigned lo, unsigned hi, bool upper) {  // their lower or upper 16 bits side by side
  return __builtin_amdgcn_perm(hi, lo, upper ? 0x07060302u : 0x05040100u);
}
// Eight columns of x as operands: bf16 rows give one, fp32 ones three whose sum is
// x, eight bits each.
template <typename T>
struct XOps;
template <>
struct XOps<uint16_t> {
  static constexpr int N = 1;
  // The weights' operand for the eight numbers of a word: 1 + q / 16, q in the upper
  // four bits of a bf16 with the exponent of 1, two numbers an operation.  The 1 and the
  // zero point are taken off by the sums of x, which the matrix unit makes from an
  // operand of ones.
  static constexpr float OFFSET = 1.f;
  static __device__ bf16x8 weights(unsigned w) {
    constexpr unsigned M = 0x00780078u, E = 0x3f803f80u;
    return words(((w << 3) & M) | E, ((w >> 1) & M) | E, ((w >> 5) & M) | E, ((w >> 9) & M) | E);
  }
  bf16x8 o[1];
  __device__ void set(const VecU<uint16_t, 8> &x) {
    o[0] = words(halves(x.v.x, x.v.z, false), halves(x.v.x, x.v.z, true), halves(x.v.y, x.v.w, false),
                 halves(x.v.y, x.v.w, true));
  }
};
template <>
struct XOps<float> {
  static constexpr int N = 3;
  // (q - 8) / 16, so that sums of 24 bits lose nothing to an offset: 1 + q / 16 as fp32
  // less 1.5.  The sums of x are needed for other zero points than 8 only.
  static constexpr float OFFSET = -0.5f;
  static __device__ bf16x8 weights(unsigned w) {
    unsigned p[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float a = __uint_as_float(((w << (19 - 4 * k)) & 0x00780000u) | 0x3f800000u) - 1.5f;
      const float b = __uint_as_float(((4 * k <= 3 ? w << (3 - 4 * k) : w >> (4 * k - 3)) & 0x00780000u) | 0x3f800000u) - 1.5f;
      p[k] = halves(__float_as_uint(a), __float_as_uint(b), true);
    }
    return words(p[0], p[1], p[2], p[3]);
  }
  bf16x8 o[3];
  __device__ void set(const VecU<float, 8> &x) {
    unsigned p[3][4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      float a = x.e[k], b = x.e[k + 4];
#pragma unroll
      for (int s = 0; s < 3; s++) {
        p[s][k] = halves(__float_as_uint(a), __float_as_uint(b), true);
        a -= __uint_as_float(__float_as_uint(a) & 0xffff0000u);
        b -= __uint_as_float(__float_as_uint(b) & 0xffff0000u);
      }
    }
#pragma unroll
    for (int s = 0; s < 3; s++) o[s] = words(p[s][0], p[s][1], p[s][2], p[s][3]);
  }
};

// The scales (or zero points) of one row of weights from a group on: 16 bytes at a
// time, since a row's lie in one or two lines that would not stay in the cache from
// step to step.
template <typename T>
struct GroupWindow {
  static constexpr int N = 16 / (int)sizeof(T);
  u32x4v v;
  __device__ void load(const T *p, int left) { v = ldu<T, N>(p, left).v; }
  __device__ float get(int i) const {
    VecU<T, N> e;
    e.v = v;
    return e.f(i);
  }
  template <int GROUPS>
  __device__ void drop() {
    constexpr int B = GROUPS * (int)sizeof(T);
    if constexpr (B == 2) {
      v[0] = __builtin_amdgcn_alignbit(v[1], v[0], 16);
      v[1] = __builtin_amdgcn_alignbit(v[2], v[1], 16);
      v[2] = __builtin_amdgcn_alignbit(v[3], v[2], 16);
      v[3] >>= 16;
    } else if constexpr (B == 4) {
      v = u32x4v{v[1], v[2], v[3], 0u};
    } else if constexpr (B == 8) {
      v = u32x4v{v[2], v[3], 0u, 0u};
    }
  }
};

// For one token or a decoding batch the weights' bytes are the floor; what they cost
// on the way is what bounds the kernel: two operations for two numbers, a transposition
// and the scales' for each group.  Few rows leave the matrix unit nearly idle (5% at 16
// rows), so its 16 rows are no waste, and it takes over the sums of x besides.  The
// scale multiplies a group's sum once and not each weight.
// Measured (bf16): one token, 4096 x 4096, groups of 128: 6.4 us, of which a launch with
// its first loads is 3 to 4; one token on 32768 x 4096, with zero points: 23; 16 rows of it,
// groups of 64: 28 us for 77 MB (2.7 TB/s; VALU issue 47% by the counters at two wavefronts
// a SIMD, whose registers are full; twice the wavefronts by two tiles of columns take 40);
// without zero points, groups of 128: 25; 64 rows, which unpack every weight four times: 83 to 86.
// MT x NT tiles of 16 rows of x by 16 columns of the output; WV wavefronts take
// slices of K, 256 columns (a line of a row of weights) at a time, and join in
// shared memory.  GM: groups in 128 columns, 1 (also where a group is several times
// 128), 2 or 4, or 0 where groups end anywhere between 32 columns.
template <typename T, int MT, int NT, int GM, int WV, bool ZERO>
__global__ __launch_bounds__(64 * WV, 2) void k_w4_rows(W4Args a) {
  constexpr int NG = GM ? GM : 4;
  constexpr bool SUMS = ZERO || XOps<T>::OFFSET != -8.f / W4_UNIT;
  __shared__ float red[WV][NT * 256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, q = lane >> 4;
  // (blocks side by side share weights: they are read from memory once)
  const int mb = (a.M + 16 * MT - 1) / (16 * MT);
  const int n0 = (int)(blockIdx.x / mb) * 16 * NT, m0 = (int)(blockIdx.x % mb) * 16 * MT;
  // rows past the end read the last one; their results are not stored
  const uint8_t *wp[NT];
  const T *xp[MT], *sp[NT], *zp[NT];
#pragma unroll
  for (int j = 0; j < NT; j++) {
    const int n = n0 + j * 16 + c < a.N ? n0 + j * 16 + c : a.N - 1;
    wp[j] = a.q + n * a.ldq + q * 16;
    sp[j] = (const T *)a.scale + (long long)n * a.G;
    zp[j] = (const T *)a.zero + (long long)n * a.G;
  }
#pragma unroll
  for (int i = 0; i < MT; i++) {
    const int m = m0 + i * 16 + c < a.M ? m0 + i * 16 + c : a.M - 1;
    xp[i] = (const T *)a.x + m * a.ldx + q * 8;
  }
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int j = 0; j < NT; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int k0 = wave * a.slice, k1 = a.K - k0 < a.slice ? a.K : k0 + a.slice;
  // the group of the 32 columns from k on (k / 32 below 2^19: the product is off by
  // less than the half that separates it from the next number)
  auto group = [&](int k) { return (int)(((float)(k >> 5) + 0.5f) * a.rgroup); };
  auto load_w = [&](u32x4v (&w)[NT][2], int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const int k = kb + W4_CH * u;
        if (k + W4_CH <= a.K) w[j][u] = reinterpret_cast<const Packed<uint8_t, 16> *>(wp[j] + (k >> 1))->v;
        else w[j][u] = ldu<uint8_t, 16>(wp[j] + (k >> 1), (a.K + 1) / 2 - (k >> 1) - q * 16).v;  // not past the row's end
      }
  };
  auto load_x = [&](VecU<T, 8> (&x)[MT][4], int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const T *p = xp[i] + kb + 32 * u;
        if (kb + W4_CH <= a.K) x[i][u].v = reinterpret_cast<const Packed<T, 8> *>(p)->v;
        else x[i][u] = ldu<T, 8>(p, a.K - kb - 32 * u - 8 * q);  // zeros past the end
      }
  };
  const bf16x8 ones = words(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  const f32x4 nil = {0.f, 0.f, 0.f, 0.f};
  // scales and zero points: from the window, or for each 32 columns
  GroupWindow<T> gs[NT], gz[NT];
  int have = 0, g0 = group(k0);                      // groups left in the window, the next one's number
  const int per = GM == 1 ? a.group / W4_CH : 1;     // steps of a group
  int stay = GM == 1 ? per - (k0 / W4_CH) % per : 1;  // steps left in this one
  auto step = [&](const u32x4v (&w)[NT][2], int half, const VecU<T, 8> (&xv)[MT][4], int kb) __attribute__((always_inline)) {
    float sc[NT][NG], zr[NT][NG];
    if constexpr (GM == 0) {
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const int g = min(group(kb + 32 * u), a.G - 1);
#pragma unroll
        for (int j = 0; j < NT; j++) {
          sc[j][u] = ldf(sp[j], g);
          zr[j][u] = ZERO ? ldf(zp[j], g) : 8.f;
        }
      }
    } else {
      if (have == 0) {
#pragma unroll
        for (int j = 0; j < NT; j++) {
          gs[j].load(sp[j] + g0, a.G - g0);
          if (ZERO) gz[j].load(zp[j] + g0, a.G - g0);
        }
        have = GroupWindow<T>::N;
        g0 += have;
      }
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int u = 0; u < NG; u++) {
          sc[j][u] = gs[j].get(u);
          zr[j][u] = ZERO ? gz[j].get(u) : 8.f;
        }
      if (--stay == 0) {
        stay = per;
        have -= NG;
#pragma unroll
        for (int j = 0; j < NT; j++) {
          gs[j].template drop<NG>();
          if (ZERO) gz[j].template drop<NG>();
        }
      }
    }
    // lane q's word j holds columns 32 q + 8 j ..; the matrix product of 32 columns
    // wants 32 j + 8 q ..: a transposition of 4 x 4 words between the lanes' rows
    unsigned b[NT][4];
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const u32x4v v = w[j][half];
      const auto e = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
      const auto f = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
      const auto g = __builtin_amdgcn_permlane16_swap(e[0], f[0], false, false);
      const auto h = __builtin_amdgcn_permlane16_swap(e[1], f[1], false, false);
      b[j][0] = g[0];
      b[j][1] = g[1];
      b[j][2] = h[0];
      b[j][3] = h[1];
    }
    f32x4 xs[MT], d[MT][NT];
#pragma unroll
    for (int u = 0; u < 4; u++) {
      bf16x8 bw[NT];
#pragma unroll
      for (int j = 0; j < NT; j++) bw[j] = XOps<T>::weights(b[j][u]);
#pragma unroll
      for (int i = 0; i < MT; i++) {
        XOps<T> x;
        x.set(xv[i][u]);
        if (u % (4 / NG) == 0) {
          xs[i] = nil;
#pragma unroll
          for (int j = 0; j < NT; j++) d[i][j] = nil;
        }
#pragma unroll
        for (int o = 0; o < XOps<T>::N; o++) {
          if (SUMS) xs[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.o[o], ones, xs[i], 0, 0, 0);
#pragma unroll
          for (int j = 0; j < NT; j++)
            d[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.o[o], bw[j], d[i][j], 0, 0, 0);
        }
        if (u % (4 / NG) == 4 / NG - 1) {
#pragma unroll
          for (int j = 0; j < NT; j++)
#pragma unroll
            for (int r = 0; r < 4; r++)
              acc[i][j][r] = fmaf(sc[j][u * NG / 4], SUMS ? fmaf(fmaf(zr[j][u * NG / 4], -1.f / W4_UNIT, -XOps<T>::OFFSET), xs[i][r], d[i][j][r]) : d[i][j][r], acc[i][j][r]);
        }
      }
    }
  };
  // the next 256 columns' weights in flight during a pair of steps, and where there
  // are registers the next step's x
  constexpr bool AHEAD = MT * NT * sizeof(T) <= 4;
  u32x4v w0[NT][2], w1[NT][2];
  VecU<T, 8> x0[MT][4], x1[MT][4];
  auto pair = [&](const u32x4v (&w)[NT][2], u32x4v (&next)[NT][2], int kb) __attribute__((always_inline)) {
    if (kb + 2 * W4_CH < k1) load_w(next, kb + 2 * W4_CH);
    if (!AHEAD) load_x(x0, kb);
    else if (kb + W4_CH < k1) load_x(x1, kb + W4_CH);
    step(w, 0, x0, kb);
    if (kb + W4_CH >= k1) return;
    if (!AHEAD) load_x(x0, kb + W4_CH);
    else if (kb + 2 * W4_CH < k1) load_x(x0, kb + 2 * W4_CH);
    step(w, 1, AHEAD ? x1 : x0, kb + W4_CH);
  };
  if (k0 < k1) {
    load_w(w0, k0);
    if (AHEAD) load_x(x0, k0);
  }
  for (int kb = k0; kb < k1; kb += 4 * W4_CH) {
    pair(w0, w1, kb);
    if (kb + 2 * W4_CH >= k1) break;
    pair(w1, w0, kb + 2 * W4_CH);
  }
#pragma unroll
  for (int i = 0; i < MT; i++) {
    if (i) __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int r = 0; r < 4; r++) red[wave][(q * 4 + r) * 16 * NT + j * 16 + c] = acc[i][j][r];
    __syncthreads();
    for (int e = threadIdx.x; e < NT * 256; e += 64 * WV) {
      const int m = m0 + i * 16 + e / (16 * NT), n = n0 + e % (16 * NT);
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < WV; w++) v += red[w][e];
      if (m < a.M && n < a.N)
        stf((T *)a.out + m * a.ldo, n, a.bias ? fmaf(v, W4_UNIT, ldf((const T *)a.bias, n)) : v * W4_UNIT);
    }
  }
}

// Tiles of a block.  A step of a tile of columns reads 1 KB of weights, one of a
// tile of bf16 rows 4 KB of x (from the L2, which holds it): columns side by side
// share x, as long as there are blocks for all CUs, and where there are many, two
// tiles of rows share weights.
struct W4Geom {
  int mt, nt;
};
static W4Geom w4_geom(int dtype, int M, int N, bool zero) {
  const long long rows = (M + 15) / 16, cols = (N + 15) / 16, tiles = rows * cols;
  const bool bf = dtype == PR_BF16;
  // (fp32 rows with zero points, which one tile of rows takes two tiles of columns
  // only: 64 x 32768 x 4096 in 173 us against 206; without zero points, and in bf16,
  // four columns are faster: 127 against 157, 86 against 117)
  if (rows > 1 && tiles >= 4 * 256 && (tiles < 8 * 256 || (!bf && zero))) return {2, 2};
  // (zero points take the registers of 2 x 4 tiles, and of 1 x 4 with fp32 rows)
  if (rows > 1 && tiles >= 8 * 256 && bf && !zero) return {2, 4};
  return {1, tiles >= 4 * 256 && (bf || !zero) ? 4 : tiles >= 2 * 256 ? 2 : 1};
}
template <typename T, int MT, int NT, bool ZERO, int WV>
void w4_groups(W4Args &a, unsigned blocks, hipStream_t s) {
  const int steps = (a.K + W4_CH - 1) / W4_CH;
  a.slice = (steps + WV - 1) / WV * W4_CH;
  if (a.group % W4_CH == 0) k_w4_rows<T, MT, NT, 1, WV, ZERO><<<blocks, 64 * WV, 0, s>>>(a);
  else if (a.group == 64) k_w4_rows<T, MT, NT, 2, WV, ZERO><<<blocks, 64 * WV, 0, s>>>(a);
  else if (a.group == 32) k_w4_rows<T, MT, NT, 4, WV, ZERO><<<blocks, 64 * WV, 0, s>>>(a);
  else k_w4_rows<T, MT, NT, 0, WV, ZERO><<<blocks, 64 * WV, 0, s>>>(a);
}
template <typename T, bool ZERO>
hipError_t w4_launch(W4Args &a, const W4Geom &g, unsigned blocks, hipStream_t s) {
  if (g.mt == 2) {
    if constexpr (sizeof(T) == 2 && !ZERO)
      if (g.nt == 4) w4_groups<T, 2, 4, ZERO, 4>(a, blocks, s);
    if (g.nt == 2) w4_groups<T, 2, 2, ZERO, 8>(a, blocks, s);
  } else if (g.nt == 4) {
    if constexpr (sizeof(T) == 2 || !ZERO) w4_groups<T, 1, 4, ZERO, 4>(a, blocks, s);
  } else if (g.nt == 2) {
    w4_groups<T, 1, 2, ZERO, 8>(a, blocks, s);
  } else {
    w4_groups<T, 1, 1, ZERO, 8>(a, blocks, s);
  }
  return hipGetLastError();
}

struct W4QuantArgs {
  void *w, *scale, *zero;  // zero may be null
  uint8_t *q;
  long long ldw, ldq;
  int N, K, group, G;
};

// y / s, correctly rounded, for s > 0 and finite.  With inv the rounded reciprocal,
// the product's exact remainder times inv corrects it, three operations for a
// division's dozen; scales near the ends of the range are divided by.
struct Divisor {
  float s, inv;
  bool plain;
  __device__ explicit Divisor(float v) : s(v), inv(__fdiv_rn(1.f, v)), plain(v > 1e-30f && v < 1e30f) {}
  __device__ float of(float y) const {
    const float q = y * inv;
    return plain ? fmaf(fmaf(-q, s, y), inv, q) : __fdiv_rn(y, s);
  }
};

// Bound by memory: 8192 x 4096 in bf16 to groups of 128 takes 21 us (84 MB, 3.9 TB/s;
// the reciprocal, the maximum over lanes and the rounding stand between a group's one
// load and one store), and back 15.8 (5.3 TB/s).
// L lanes (a power of two) for each group, eight columns each, which stay in
// registers between the extremes and the rounding; groups of more than 8 L columns
// (L = 64) are read again.
template <typename T, int L, bool ZERO>
__global__ __launch_bounds__(256) void k_w4_quant(W4QuantArgs a) {
  const long long id = flat_block() * (256 / L) + threadIdx.x / L;  // row and group
  const int lane = threadIdx.x % L;
  const bool on = id < (long long)a.N * a.G;
  const int g = on ? (int)(id % a.G) : 0;
  const long long n = on ? id / a.G : 0;
  const int k0 = g * a.group, k1 = on ? (a.K - k0 < a.group ? a.K : k0 + a.group) : k0, first = k0 + lane * 8;
  const T *wp = (const T *)a.w + n * a.ldw;
  const VecU<T, 8> own = ldu<T, 8>(wp + first, k1 - first);
  // the largest of max(w, 0) and of max(-w, 0), compared by their bits: a NaN wins
  unsigned hi = 0, lo = 0;
  auto extremes = [&](const VecU<T, 8> &v) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float f = v.f(i);
      const unsigned bits = __float_as_uint(fabsf(f)), up = !ZERO || f > 0.f || f != f ? bits : 0u;
      hi = max(hi, up);
      if (ZERO) lo = max(lo, bits ^ up);
    }
  };
  extremes(own);
  if constexpr (L == 64)
    for (int k = first + L * 8; k < k1; k += L * 8) extremes(ldu<T, 8>(wp + k, k1 - k));
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) {
    hi = max(hi, (unsigned)__shfl_xor((int)hi, o, 64));
    if (ZERO) lo = max(lo, (unsigned)__shfl_xor((int)lo, o, 64));
  }
  const float fh = __uint_as_float(hi), fl = __uint_as_float(lo);
  T st;
  stf(&st, 0, ZERO ? (fh + fl) * (1.f / 15.f) : fh * (1.f / 7.f));
  const float s = ldf(&st, 0);
  const bool some = s > 0.f && s < __builtin_inff();
  const Divisor by(some ? s : 1.f);
  float z = 8.f;
  if (ZERO) z = some ? fminf(fmaxf(rintf(by.of(fl)), 0.f), 15.f) : s == 0.f ? 0.f : 8.f;
  if (on && lane == 0) {
    ((T *)a.scale)[id] = st;
    if (ZERO) stf((T *)a.zero, id, z);
  }
  auto store = [&](int k, const VecU<T, 8> &v) {
    const int c = k1 - k;
    // held to the range, then rounded by the sum with 1.5 2^23, whose bits are a
    // constant plus the number; constants and the zero point come off the whole word
    unsigned word = ((unsigned)(int)z - 0x4b400000u) * 0x11111111u;
    const float low = -z, high = 15.f - z;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float f = some ? __builtin_amdgcn_fmed3f(by.of(v.f(i)), low, high) : 0.f;
      word += __float_as_uint(f + 12582912.f) << (4 * i);
    }
    uint8_t *qp = a.q + n * a.ldq + (k >> 1);
    if (c >= 8) {
      reinterpret_cast<Packed<uint8_t, 4> *>(qp)->v = word;
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (2 * i < c) qp[i] = (uint8_t)(word >> (8 * i));
    }
  };
  if (first < k1) store(first, own);
  if constexpr (L == 64)
    for (int k = first + L * 8; k < k1; k += L * 8) store(k, ldu<T, 8>(wp + k, k1 - k));
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
    const dim3 grid = flat_grid((groups * L + 255) / 256);                         \
    if (a.zero) k_w4_quant<T, L, true><<<grid, 256, 0, s>>>(a);                    \
    else k_w4_quant<T, L, false><<<grid, 256, 0, s>>>(a);                          \
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

int w4_group_count(int K, int group) { return (int)(((long long)K + group - 1) / group); }

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
  a.ldx = ldx; a.ldq = ldq; a.ldo = ldo; a.M = M; a.N = N; a.K = K; a.group = group; a.G = w4_group_count(K, group);
  a.rgroup = 32.f / (float)group;
  const W4Geom g = w4_geom(dtype, M, N, zero != nullptr);
  const long long blocks = (long long)((N + 16 * g.nt - 1) / (16 * g.nt)) * ((M + 16 * g.mt - 1) / (16 * g.mt));
  // a launch has 2^32 threads at most, 512 a block
  if (blocks >= (1 << 23)) return fail(PR_EUNSUPPORTED, "problem too large: %d x %d results", M, N);
  hipStream_t s = (hipStream_t)stream;
  const unsigned nb = (unsigned)blocks;
  if (dtype == PR_BF16) HIPCHK((zero ? w4_launch<uint16_t, true>(a, g, nb, s) : w4_launch<uint16_t, false>(a, g, nb, s)));
  else HIPCHK((zero ? w4_launch<float, true>(a, g, nb, s) : w4_launch<float, false>(a, g, nb, s)));
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
  W4QuantArgs a{(void *)w, scale, zero, q, ldw, ldq, N, K, group, w4_group_count(K, group)};
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
  W4QuantArgs a{w, (void *)scale, (void *)zero, (uint8_t *)q, ldw, ldq, N, K, group, w4_group_count(K, group)};
  const int per = (K + 7) / 8;
  const dim3 grid = flat_grid(((long long)N * per + 255) / 256);
  if (dtype == PR_BF16) k_w4_dequant<uint16_t><<<grid, 256, 0, (hipStream_t)stream>>>(a, per);
  else k_w4_dequant<float><<<grid, 256, 0, (hipStream_t)stream>>>(a, per);
  HIPCHK(hipGetLastError());
  return PR_OK;
}

}  // extern "C"
