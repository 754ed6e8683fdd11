// Gated linear recurrence, its adjoint and its single-token step.
//
//   r = sigm(rg + rb), i = sigm(ig + ib), v = decay r, a = e^-v,
//   m = sqrt(1 - a^2), h_t = a h_{t-1} + m i x_t
// Adjoint, with g_t = dy_t + a_{t+1} g_{t+1}:
//   dx = g m i, di = g m x i (1 - i), dv = g (a^2 / m i x - a h_{t-1}),
//   dr = dv decay r (1 - r), ddecay = sum dv r
//
// Bound by memory, with instruction issue close behind.  A step is an affine map of
// the state, h -> a h + m i x, and maps compose: B ceil(D / 64) columns alone leave
// most of the device idle (4 of them in one sequence of 256 channels), so time is cut
// into tiles that run side by side and are joined in the same pass, each input read
// once.  Two passes, one for the tiles' maps and one for their steps, would read
// the three inputs twice.  The adjoint reads x, r and i
// again and makes the gates and states anew: storing a, m and both gates in fp32 would
// move 32 bytes a step and channel to save 4.
// Measured: 8 x 4096 x 2048, bf16, forward with saved states 125 us for 550 MB (4.4
// TB/s, VALU issue 64% by the counters), adjoint 264 us for 976 MB (3.7 TB/s, 62%; three
// outputs and four inputs share the memory's reads and writes, and at three wavefronts a
// SIMD a tile's phases, load, gates, join, walk and store, do not fill each other's
// gaps), the sums of decay's and the biases' gradients 8, the chains' clearing 5 to 6
// each; 1 x 32768 x 256, fp32, 35 us (3.9 TB/s: 2048 tiles, of which each waits for
// those before it); 4 x 4096 x 2048, fp32, training 306 us together.
#include <type_traits>

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
  int cb, tiles, tt, nst;    // columns of channels a sequence, tiles a column, steps a tile, saved states a sequence
};

// What a step's gates give: both gates, and a = e^-v, its logarithm l (SHORT: to base
// 2) and m = sqrt(1 - a^2) for v = decay r.
struct GateVals {
  float r, i, a, l, m;
};
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
// A channel's constants.  Rows stored in 8 significant bits take plain products
// for the exponentials' arguments, with the constants folded in; fp32 ones carry
// the products in two words.
template <typename T>
struct GateConsts {
  static constexpr bool SHORT = sizeof(T) == 2;
  float rb, ib, nd;  // nd = -decay; SHORT: the biases and the decay times -log2 e
  __device__ GateConsts(float decay, float r_bias, float i_bias)
      : rb(SHORT ? -LOG2E * r_bias : r_bias), ib(SHORT ? -LOG2E * i_bias : i_bias), nd(SHORT ? -LOG2E * decay : -decay) {}
};
template <typename T>
__device__ inline GateVals gate_vals(float rg, float ig, const GateConsts<T> &c) {
  GateVals o;
  if constexpr (GateConsts<T>::SHORT) {
    o.r = frcp(1.f + __builtin_amdgcn_exp2f(fmaf(rg, -LOG2E, c.rb)));
    o.i = frcp(1.f + __builtin_amdgcn_exp2f(fmaf(ig, -LOG2E, c.ib)));
    o.l = c.nd * o.r;
    o.a = __builtin_amdgcn_exp2f(o.l);
  } else {
    o.r = frcp(1.f + exp_any(-(rg + c.rb)));
    o.i = frcp(1.f + exp_any(-(ig + c.ib)));
    o.l = c.nd * o.r;
    o.a = exp_acc(o.l);
  }
  // 1 - e^-w for w = 2 v: the difference where little is lost, else its series.
  // SHORT: up to w^4, the first term left out is below w^4 / 120 of it, 1.3e-7 at
  // w = 1/16, where the difference has lost 4 bits; else up to w^6, 5e-8 at 1/4.
  const float w = o.l * (GateConsts<T>::SHORT ? -2.f * LN2 : -2.f);
  float s;
  if constexpr (GateConsts<T>::SHORT) {
    s = fmaf(w, -1.f / 24.f, 1.f / 6.f);
  } else {
    s = fmaf(w, -1.f / 720.f, 1.f / 120.f);
    s = fmaf(w, s, -1.f / 24.f);
    s = fmaf(w, s, 1.f / 6.f);
  }
  s = fmaf(w, s, -0.5f);
  s = fmaf(w, s, 1.f);
  o.m = __builtin_amdgcn_sqrtf(w < (GateConsts<T>::SHORT ? 0.0625f : 0.25f) ? w * s : fmaf(-o.a, o.a, 1.f));
  return o;
}

// A sequence of steps multiplies the state by e^(sum of their l).  Near 1 a factor in
// fp32 is off by a part of 1 - a that may be large, the same at every step of a steady
// gate, and a product of thousands of them by thousands of times that (1e-3 of a state
// kept over 24000 steps); the sum keeps what a factor loses.  So longer runs of steps
// go by their sum, to base 2.
__device__ inline float decay_of(float l2) { return __builtin_amdgcn_exp2f(l2); }
// A h + b for A = e^-v, without the factor's rounding: near 1 by what it takes off,
// 1 - e^-v, whose series is that of m^2.  (An infinite state takes the product.)
__device__ inline float decayed(float A, float v, float h, float b) {
  float s = fmaf(v, -1.f / 24.f, 1.f / 6.f);
  s = fmaf(v, s, -0.5f);
  s = fmaf(v, s, 1.f);
  const float e = v < 0.0625f ? v * s : 1.f - A, near = h + fmaf(-e, h, b);
  return A > 0.5f && near == near ? near : fmaf(A, h, b);
}
__device__ inline float decayed(float l2, float h, float b) { return decayed(decay_of(l2), l2 * -LN2, h, b); }

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
// A block takes 64 channels (a column of tiles) and a tile of steps: a lane
// holds four adjacent channels, a wavefront four rows of K steps each.  Every
// lane composes its steps, one wavefront joins the rows and the tiles before,
// and every lane then walks its steps again from its row's state, so that each
// input is read once.
constexpr int G_CH = 64;
constexpr int G_SUPER = 8;  // tiles of a super tile

// State between the tiles of a column.  A tile publishes what it does to a
// state, h -> 2^L h + B; the last of 8 publishes the same of all 8, and, once it
// is known, the state that leaves them.  A tile's state is the one that enters
// its super tile, taken through the tiles before it in order, and that one is
// the first state, taken through the super tiles in order: the same products and
// sums whatever was published when it looked, so results repeat bit by bit.
//   Words of 64 bits, L or 0 above B or the state; all ones: not there yet.  The
// word is read and written whole, so nothing has to be ordered around it.
//   Tiles of a column are handed out in order by a counter: a tile waits only for
// blocks that already run, whatever else runs on the device.
struct GatedChain {
  unsigned *ticket;                        // [columns], 64 bytes apart
  unsigned long long *agg, *sagg, *spre;   // [tile][column][64], [super][column][64], [super][column][64]
  long long cols;
};
constexpr unsigned G_NONE = 0xffffffffu;
__device__ inline unsigned long long chain_word(float L, float B) {
  const unsigned h = __float_as_uint(L);
  return ((unsigned long long)(h == G_NONE ? 0x7fc00000u : h) << 32) | __float_as_uint(B);
}
__device__ inline bool chain_there(unsigned long long w) { return (unsigned)(w >> 32) != G_NONE; }
__device__ inline float chain_L(unsigned long long w) { return __uint_as_float((unsigned)(w >> 32)); }
__device__ inline float chain_B(unsigned long long w) { return __uint_as_float((unsigned)w); }

// The state that enters tile j (j-th in the order of the chain) of column c,
// for one channel a lane, after the tile's own L, B were published; `first`: the
// column's first state, read by tile 0 alone.  A wait that sees nothing for
// PR_SPIN_LIMIT polls gives up with a NaN.
__device__ inline float chain_enter(const GatedChain &ch, long long c, int j, int tiles, float L, float B, float first) {
  const unsigned lane = threadIdx.x & 63;
  const int s = j / G_SUPER, q = j % G_SUPER;
  const long long step = ch.cols * 64;
  unsigned long long *agg = ch.agg + (s * (G_SUPER * step) + c * 64 + lane), *sagg = ch.sagg + (s * step + c * 64 + lane),
                     *spre = ch.spre + (s * step + c * 64 + lane);
  unsigned long long w[G_SUPER - 1], p;
  int polls = 0;
  if (j == 0) {
    if (tiles > 1) st_agent64(spre, chain_word(0.f, first));
    return first;
  }
  while (true) {
    bool ok = true;
    long long st = step;
    asm volatile("" : "+s"(st));  // addresses made where they are used: kept over the loop they would take 60 registers
#pragma unroll
    for (int i = 0; i < G_SUPER - 1; i++)
      if (i < q) w[i] = ld_agent64(agg + i * st);
    p = ld_agent64(spre);
#pragma unroll
    for (int i = 0; i < G_SUPER - 1; i++)
      if (i < q) ok = ok && chain_there(w[i]);
    if (__all(ok)) break;
    if (++polls > PR_SPIN_LIMIT) return __builtin_nanf("");
    __builtin_amdgcn_s_sleep(1);
  }
  float SL = L, SB = B;
  const bool closes = q == G_SUPER - 1 && j + 1 < tiles;
  if (closes) {
    SL = chain_L(w[0]);
    SB = chain_B(w[0]);
#pragma unroll
    for (int i = 1; i < G_SUPER - 1; i++) {
      SB = fmaf(decay_of(chain_L(w[i])), SB, chain_B(w[i]));
      SL += chain_L(w[i]);
    }
    SB = fmaf(decay_of(L), SB, B);
    SL += L;
    st_agent64(sagg, chain_word(SL, SB));
  }
  // the state that enters the super tile: there, or from one of the 4 before it
  float h;
  while (true) {
    constexpr int W = 4;
    bool ok = chain_there(p);
    h = chain_B(p);
    if (__all(ok)) break;
    unsigned long long pre[W], ag[W];
    long long st = step;
    asm volatile("" : "+s"(st));
#pragma unroll
    for (int i = 0; i < W; i++)
      if (s - 1 - i >= 0) {
        pre[i] = ld_agent64(spre - (i + 1) * st);
        ag[i] = ld_agent64(sagg - (i + 1) * st);
      } else {
        pre[i] = ag[i] = ~0ull;
      }
    int from = -1;  // the nearest state that was published, with all that follows it
    bool all = true;
#pragma unroll
    for (int i = 0; i < W; i++) {
      all = all && chain_there(ag[i]);
      if (from < 0 && all && chain_there(pre[i])) from = i;
    }
    float v = 0.f;
#pragma unroll
    for (int i = W - 1; i >= 0; i--) {
      if (i == from) v = chain_B(pre[i]);
      if (i <= from) v = decayed(chain_L(ag[i]), v, chain_B(ag[i]));
    }
    if (!ok) {
      ok = from >= 0;
      h = v;
    }
    if (__all(ok)) break;
    if (++polls > PR_SPIN_LIMIT) return __builtin_nanf("");
    __builtin_amdgcn_s_sleep(1);
    p = ld_agent64(spre);
  }
  if (closes) st_agent64(spre + step, chain_word(0.f, decayed(SL, h, SB)));
#pragma unroll
  for (int i = 0; i < G_SUPER - 1; i++)
    if (i < q) h = fmaf(decay_of(chain_L(w[i])), h, chain_B(w[i]));
  return h;
}

__global__ __launch_bounds__(256) void k_gated_clear(uint4 *p, long long n) {
  for (long long i = flat_block() * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * gridDim.y * 256)
    p[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

// A tile's steps of one [B, T, D] array: the tile's first step (uniform), with
// 32-bit offsets of at most 128 steps from it.
struct TileOf {
  char *base;
  unsigned st;  // bytes
};
template <typename T>
__device__ inline TileOf tile_of(const View &v, int b, long long t0) {
  return TileOf{(char *)((T *)v.p + b * v.sb + t0 * v.st), (unsigned)v.st * (unsigned)sizeof(T)};
}

// Where a lane stands.
struct GatedAt {
  int d, n;     // first channel, channels from it on
  int t0, row;  // the tile's first step, the lane's first step in it
  int len;      // steps of the sequence
};
// Four channels of the K steps of a lane in N arrays, all loads in flight
// together.  Not FULL: steps past the end read the last one, lanes past the last
// channel others of the row, whose values nobody uses.
template <typename T, bool FULL, int K, int N>
__device__ inline void ld_steps(const TileOf (&v)[N], const GatedAt &p, int D, VecU<T, 4> (&r)[N][K]) {
  if (FULL || D >= 4) {
    const int dd = FULL || p.d < D - 4 ? p.d : D - 4, m = p.d - dd, last = p.len - 1 - p.t0;
#pragma unroll
    for (int k = 0; k < K; k++) {
      const int s = FULL || p.row + k < last ? p.row + k : last;
#pragma unroll
      for (int j = 0; j < N; j++) {
        // (FULL: one offset for all steps of an array)
        const unsigned off = (unsigned)(FULL ? p.row : s) * v[j].st + (unsigned)dd * (unsigned)sizeof(T);
        r[j][k].v = reinterpret_cast<const Packed<T, 4> *>(v[j].base + (FULL ? (long long)k * v[j].st : 0) + off)->v;
      }
    }
    if constexpr (!FULL)
#pragma unroll
      for (int k = 0; k < K; k++)
#pragma unroll
        for (int j = 0; j < N; j++) {
          VecU<T, 4> &e = r[j][k];
          const T e1 = e.e[1], e2 = e.e[2], e3 = e.e[3];
          e.e[0] = m == 0 ? e.e[0] : m == 1 ? e1 : m == 2 ? e2 : e3;
          e.e[1] = m == 0 ? e1 : m == 1 ? e2 : e3;
          e.e[2] = m == 0 ? e2 : e3;
        }
  } else {
    const int last = p.len - 1 - p.t0;
#pragma unroll
    for (int k = 0; k < K; k++)
#pragma unroll
      for (int j = 0; j < N; j++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const unsigned off = (unsigned)(p.row + k < last ? p.row + k : last) * v[j].st;
          r[j][k].e[i] = reinterpret_cast<const T *>(v[j].base + off)[p.d + i < D ? p.d + i : D - 1];
        }
  }
}
template <typename T, bool FULL>
__device__ inline void st_step(const TileOf &v, const GatedAt &p, int k, int T_, const float *o) {
  const unsigned off = (unsigned)p.row * v.st + (unsigned)p.d * (unsigned)sizeof(T);
  T *q = (T *)(v.base + (long long)k * v.st + off);
  if constexpr (FULL) stu_nt<T, 4>(q, o, 4);
  else if (p.t0 + p.row + k < T_ && p.n > 0) stu<T, 4>(q, o, p.n);
}
template <typename T>
__device__ inline void zero_steps(const View &v, int b, const GatedAt &p, int K, int T_) {
  const float z[4] = {0.f, 0.f, 0.f, 0.f};
  if (v.p)
    for (int k = 0; k < K; k++) st_step<T, false>(tile_of<T>(v, b, p.t0), p, k, T_, z);
}

template <typename T>
struct Consts4 {
  GateConsts<T> c[4];
};
template <typename T>
__device__ inline Consts4<T> gated_consts(const float *decay, const float *rb, const float *ib, int d, int n) {
  const VecU<float, 4> e = ldu<float, 4>(decay + d, n), r = ldu<float, 4>(rb + d, rb ? n : 0),
                       i = ldu<float, 4>(ib + d, ib ? n : 0);
  return {{{e.f(0), r.f(0), i.f(0)}, {e.f(1), r.f(1), i.f(1)}, {e.f(2), r.f(2), i.f(2)}, {e.f(3), r.f(3), i.f(3)}}};
}

// The block's column and tile (in the order of the chain); false: none left.
__device__ inline bool gated_tile(const GatedArgs &a, const GatedChain &ch, int *sh, long long *c, int *j) {
  const long long blk = flat_block();
  if (blk >= ch.cols * a.tiles) return false;
  // blocks go to the eight XCDs in turn: one XCD takes columns side by side, whose
  // pieces of a row meet in its cache and in memory (8 x 4096 x 2048: 8 and 3 %)
  *c = blk % ch.cols;
  if (ch.cols % 8 == 0) *c = (*c % 8) * (ch.cols / 8) + *c / 8;
  *j = 0;
  if (a.tiles > 1) {
    if (threadIdx.x == 0) *sh = (int)(add_agent(ch.ticket + *c * 16, 1u) + 1u);  // (starts at all ones)
    __syncthreads();
    *j = __builtin_amdgcn_readfirstlane(*sh);
  }
  return true;
}

template <typename T, int K, int NW, int WPS>
__global__ __launch_bounds__(64 * NW, WPS) void k_gated_fwd(GatedArgs a, GatedChain ch) {
  // of each row of steps: its factor, its sum B (then its first state), its factor's logarithm
  __shared__ __attribute__((aligned(16))) float lA[4 * NW * G_CH], lB[4 * NW * G_CH], lL[4 * NW * G_CH];
  __shared__ int sh;
  long long c;
  int tile;
  if (!gated_tile(a, ch, &sh, &c, &tile)) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nw = blockDim.x >> 6;
  const int b = (int)(c / a.cb), d0 = (int)(c % a.cb) * G_CH;
  const int len = __builtin_amdgcn_readfirstlane(seq_len(a.lengths, b, a.T));
  const int live = len > 0 ? (len - 1) / a.tt + 1 : 0;  // tiles of the sequence that hold steps
  const bool owns = w == 0 && d0 + lane < a.D;  // wavefront 0 joins: a lane for each channel
  const long long sd = (long long)b * a.D + d0 + lane;
  float first = 0.f;
  if (tile == 0 && a.h0 && owns) first = a.h0[sd];
  GatedAt p;
  p.d = d0 + (lane & 15) * 4;
  p.n = a.D - p.d;
  p.len = len;
  p.t0 = tile * a.tt;
  p.row = (w * 4 + (lane >> 4)) * K;
  if (tile >= live) {
    zero_steps<T>(a.y, b, p, K, a.T);
    if (tile == 0 && a.hlast && owns) a.hlast[sd] = first;
    return;
  }
  auto body = [&](auto full) __attribute__((always_inline)) {
    constexpr bool FULL = decltype(full)::value;
    float ga[K][4], gb[K][4], L[4], B[4];
    {
      const TileOf in[3] = {tile_of<T>(a.r, b, p.t0), tile_of<T>(a.i, b, p.t0), tile_of<T>(a.x, b, p.t0)};
      VecU<T, 4> raw[3][K];
      ld_steps<T, FULL, K>(in, p, a.D, raw);
      const Consts4<T> cs = gated_consts<T>(a.decay, a.rb, a.ib, p.d, p.n);
#pragma unroll
      for (int k = 0; k < K; k++) {
        const bool on = FULL || p.t0 + p.row + k < len;
#pragma unroll
        for (int v = 0; v < 4; v++) {
          const GateVals g = gate_vals<T>(raw[0][k].f(v), raw[1][k].f(v), cs.c[v]);
          ga[k][v] = on ? g.a : 1.f;
          gb[k][v] = on ? g.m * g.i * raw[2][k].f(v) : 0.f;
          L[v] = (k ? L[v] : 0.f) + (on ? g.l : 0.f);
          B[v] = k ? fmaf(ga[k][v], B[v], gb[k][v]) : gb[k][v];
        }
        __builtin_amdgcn_sched_barrier(0);  // one step's temporaries at a time
      }
#pragma unroll
      for (int v = 0; v < 4; v++) L[v] *= GateConsts<T>::SHORT ? 1.f : LOG2E;
    }
    const int at = (w * 4 + (lane >> 4)) * G_CH + (lane & 15) * 4;
    *reinterpret_cast<float4 *>(lA + at) =
        make_float4(decay_of(L[0]), decay_of(L[1]), decay_of(L[2]), decay_of(L[3]));
    *reinterpret_cast<float4 *>(lB + at) = make_float4(B[0], B[1], B[2], B[3]);
    *reinterpret_cast<float4 *>(lL + at) = make_float4(L[0], L[1], L[2], L[3]);
    lds_barrier();
    if (w == 0) {
      const int rows = nw * 4;
      float h = first;
      if (live > 1) {
        float tL = lL[lane], tB = lB[lane];
#pragma unroll 3
        for (int q = 1; q < rows; q++) {
          tB = fmaf(lA[q * G_CH + lane], tB, lB[q * G_CH + lane]);
          tL += lL[q * G_CH + lane];
        }
        if (tile + 1 < live) st_agent64(ch.agg + (tile * ch.cols + c) * 64 + (unsigned)lane, chain_word(tL, tB));
        h = chain_enter(ch, c, tile, live, tL, tB, first);
      }
#pragma unroll 4
      for (int q = 0; q < rows; q++) {
        const float qa = lA[q * G_CH + lane], qb = lB[q * G_CH + lane];
        lB[q * G_CH + lane] = h;
        h = fmaf(qa, h, qb);
      }
      if (tile + 1 == live && a.hlast && owns) a.hlast[sd] = h;
    }
    lds_barrier();
    const float4 h4 = *reinterpret_cast<const float4 *>(lB + at);
    float h[4] = {h4.x, h4.y, h4.z, h4.w};
    const int t = p.t0 + p.row;
    if (a.states && t % PR_GATED_STATE_STEPS == 0 && t < len && p.n > 0)
      stu<float, 4>(a.states + ((long long)b * a.nst + t / PR_GATED_STATE_STEPS) * a.D + p.d, h, p.n);
    const TileOf ty = tile_of<T>(a.y, b, p.t0);
#pragma unroll
    for (int k = 0; k < K; k++) {
      float o[4];
#pragma unroll
      for (int v = 0; v < 4; v++) {
        h[v] = fmaf(ga[k][v], h[v], gb[k][v]);
        o[v] = FULL || t + k < len ? h[v] : 0.f;
      }
      st_step<T, FULL>(ty, p, k, a.T, o);
    }
  };
  if ((tile + 1) * (long long)a.tt <= len && d0 + G_CH <= a.D) body(std::integral_constant<bool, true>{});
  else body(std::integral_constant<bool, false>{});
}

// The adjoint, tiles from the last to the first.  mu is what the steps after a
// step add to its state's gradient: mu_{t-1} = a_t (dy_t + mu_t), the same A as
// forwards.  The tile's states are made again from the saved one.
template <typename T, int K, int NW, int WPS>
__global__ __launch_bounds__(64 * NW, WPS) void k_gated_adj(GatedArgs a, GatedChain ch) {
  __shared__ __attribute__((aligned(16))) float lds[3][4 * NW * G_CH], lL[4 * NW * G_CH];
  __shared__ float4 lcv[K][64 * NW];  // dv = g cv
  __shared__ int sh;
  float *lA = lds[0], *lF = lds[1], *lR = lds[2];
  long long c;
  int order;
  if (!gated_tile(a, ch, &sh, &c, &order)) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nw = blockDim.x >> 6;
  const int rows = nw * 4, tile = a.tiles - 1 - order;
  const int b = (int)(c / a.cb), d0 = (int)(c % a.cb) * G_CH;
  const int len = __builtin_amdgcn_readfirstlane(seq_len(a.lengths, b, a.T));
  const int live = len > 0 ? (len - 1) / a.tt + 1 : 0;
  float *part = a.part ? a.part + ((long long)b * a.tiles + tile) * 3 * a.D + d0 : nullptr;
  const int j = live - 1 - tile;  // place in the chain
  const bool on = d0 + lane < a.D;
  const long long sd = (long long)b * a.D + d0 + lane;
  float first = 0.f, start = 0.f;  // wavefront 0 joins back in time, the last one forwards: a lane for each channel
  if (w == 0 && (j == 0 || (tile == 0 && live == 0)) && a.dhlast && on) first = a.dhlast[sd];
  if (w == nw - 1 && on && tile < live)
    start = a.states[((long long)b * a.nst + (long long)tile * a.tt / PR_GATED_STATE_STEPS) * a.D + d0 + lane];
  GatedAt p;
  p.d = d0 + (lane & 15) * 4;
  p.n = a.D - p.d;
  p.len = len;
  p.t0 = tile * a.tt;
  p.row = (w * 4 + (lane >> 4)) * K;
  if (tile >= live) {
    zero_steps<T>(a.dx, b, p, K, a.T);
    zero_steps<T>(a.dr, b, p, K, a.T);
    zero_steps<T>(a.di, b, p, K, a.T);
    if (part)
      for (int q = threadIdx.x; q < 3 * G_CH; q += 64 * nw)
        if (d0 + q % G_CH < a.D) part[(long long)(q / G_CH) * a.D + q % G_CH] = 0.f;
    if (tile == 0 && w == 0 && on && a.dh0) a.dh0[sd] = first;
    return;
  }
  const int at = (w * 4 + (lane >> 4)) * G_CH + (lane & 15) * 4;
  float sums[3][4] = {};
  auto body = [&](auto full) __attribute__((always_inline)) {
    constexpr bool FULL = decltype(full)::value;
    float ga[K][4], gm[K][4], gr[K][4], gi[K][4], L[4], F[4];
    VecU<T, 4> x[K], gy[K];
    {
      const TileOf in[4] = {tile_of<T>(a.r, b, p.t0), tile_of<T>(a.i, b, p.t0), tile_of<T>(a.x, b, p.t0),
                            tile_of<T>(a.y, b, p.t0)};
      VecU<T, 4> raw[4][K];
      ld_steps<T, FULL, K>(in, p, a.D, raw);
#pragma unroll
      for (int k = 0; k < K; k++) {
        x[k] = raw[2][k];
        gy[k] = raw[3][k];
      }
      const Consts4<T> cs = gated_consts<T>(a.decay, a.rb, a.ib, p.d, p.n);
#pragma unroll
      for (int k = 0; k < K; k++) {
        const bool on = FULL || p.t0 + p.row + k < len;
#pragma unroll
        for (int v = 0; v < 4; v++) {
          const GateVals g = gate_vals<T>(raw[0][k].f(v), raw[1][k].f(v), cs.c[v]);
          if (!on) x[k].e[v] = gy[k].e[v] = 0;
          ga[k][v] = on ? g.a : 1.f;  // a step that is not there keeps mu and the state, and has no gradients
          gm[k][v] = on ? g.m : 0.f;
          gr[k][v] = on ? g.r : 0.f;
          gi[k][v] = on ? g.i : 0.f;
          const float bb = gm[k][v] * gi[k][v] * x[k].f(v);
          L[v] = (k ? L[v] : 0.f) + (on ? g.l : 0.f);
          F[v] = k ? fmaf(ga[k][v], F[v], bb) : bb;
        }
        __builtin_amdgcn_sched_barrier(0);  // one step's temporaries at a time
      }
#pragma unroll
      for (int v = 0; v < 4; v++) L[v] *= GateConsts<T>::SHORT ? 1.f : LOG2E;
    }
    float R[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = K - 1; k >= 0; k--)
#pragma unroll
      for (int v = 0; v < 4; v++) R[v] = ga[k][v] * (gy[k].f(v) + R[v]);
    // (the inputs stay as they were stored: unpacked they would take twice the registers)
#pragma unroll
    for (int k = 0; k < K; k++) asm volatile("" : "+v"(x[k].v), "+v"(gy[k].v));
    *reinterpret_cast<float4 *>(lA + at) =
        make_float4(decay_of(L[0]), decay_of(L[1]), decay_of(L[2]), decay_of(L[3]));
    *reinterpret_cast<float4 *>(lL + at) = make_float4(L[0], L[1], L[2], L[3]);
    *reinterpret_cast<float4 *>(lF + at) = make_float4(F[0], F[1], F[2], F[3]);
    *reinterpret_cast<float4 *>(lR + at) = make_float4(R[0], R[1], R[2], R[3]);
    lds_barrier();
    if (w == nw - 1) {
      float h = start;
#pragma unroll 4
      for (int q = 0; q < rows; q++) {
        const float qa = lA[q * G_CH + lane], qb = lF[q * G_CH + lane];
        lF[q * G_CH + lane] = h;
        h = fmaf(qa, h, qb);
      }
    }
    if (w == 0) {
      float mu = first;
      if (live > 1) {
        float tL = lL[(rows - 1) * G_CH + lane], tB = lR[(rows - 1) * G_CH + lane];
#pragma unroll 3
        for (int q = rows - 2; q >= 0; q--) {
          tB = fmaf(lA[q * G_CH + lane], tB, lR[q * G_CH + lane]);
          tL += lL[q * G_CH + lane];
        }
        if (j + 1 < live) st_agent64(ch.agg + (j * ch.cols + c) * 64 + (unsigned)lane, chain_word(tL, tB));
        mu = chain_enter(ch, c, j, live, tL, tB, first);
      }
#pragma unroll 4
      for (int q = rows - 1; q >= 0; q--) {
        const float qa = lA[q * G_CH + lane], qb = lR[q * G_CH + lane];
        lR[q * G_CH + lane] = mu;
        mu = fmaf(qa, mu, qb);
      }
      if (tile == 0 && a.dh0 && on) a.dh0[sd] = mu;
    }
    lds_barrier();
    // (the inputs stay as they were stored: unpacked they would take twice the registers)
#pragma unroll
    for (int k = 0; k < K; k++) asm volatile("" : "+v"(x[k].v), "+v"(gy[k].v));
    const float4 h4 = *reinterpret_cast<const float4 *>(lF + at), m4 = *reinterpret_cast<const float4 *>(lR + at);
    float h[4] = {h4.x, h4.y, h4.z, h4.w}, mu[4] = {m4.x, m4.y, m4.z, m4.w};
    // forwards through the lane's steps; m becomes m i
#pragma unroll
    for (int k = 0; k < K; k++) {
      float cv[4];
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const float m = gm[k][v], u = gi[k][v] * x[k].f(v), a1 = ga[k][v];
        cv[v] = a1 * fmaf(a1 * (m > 0.f ? frcp(m) : 0.f), u, -h[v]);
        h[v] = fmaf(a1, h[v], m * u);
        gm[k][v] = m * gi[k][v];
      }
      lcv[k][threadIdx.x] = make_float4(cv[0], cv[1], cv[2], cv[3]);  // (read by this lane alone)
    }
    const VecU<float, 4> decay = ldu<float, 4>(a.decay + p.d, p.n);
    const TileOf ox_ = tile_of<T>(a.dx, b, p.t0), or_ = tile_of<T>(a.dr, b, p.t0), oi_ = tile_of<T>(a.di, b, p.t0);
#pragma unroll
    for (int k = K - 1; k >= 0; k--) {
      const bool on = FULL || p.t0 + p.row + k < len;  // (in this step)
      float ox[4], orr[4], oi[4];
      const float4 c4 = lcv[k][threadIdx.x];
      const float cv[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const float g = gy[k].f(v) + mu[v], dv = on ? g * cv[v] : 0.f, r = gr[k][v], i = gi[k][v];
        ox[v] = on ? g * gm[k][v] : 0.f;
        oi[v] = ox[v] * x[k].f(v) * (1.f - i);
        orr[v] = dv * decay.f(v) * (r * (1.f - r));
        sums[0][v] = fmaf(dv, r, sums[0][v]);
        sums[1][v] += orr[v];
        sums[2][v] += oi[v];
        mu[v] = ga[k][v] * g;
      }
      if (a.dx.p) st_step<T, FULL>(ox_, p, k, a.T, ox);
      if (a.dr.p) st_step<T, FULL>(or_, p, k, a.T, orr);
      if (a.di.p) st_step<T, FULL>(oi_, p, k, a.T, oi);
    }
  };
  if ((tile + 1) * (long long)a.tt <= len && d0 + G_CH <= a.D) body(std::integral_constant<bool, true>{});
  else body(std::integral_constant<bool, false>{});
  if (!part) return;
  lds_barrier();  // the rows' states have been read
#pragma unroll
  for (int s = 0; s < 3; s++)
    *reinterpret_cast<float4 *>(lds[s] + at) = make_float4(sums[s][0], sums[s][1], sums[s][2], sums[s][3]);
  lds_barrier();
  for (int q = threadIdx.x; q < 3 * G_CH; q += 64 * nw) {
    float v = 0.f;
    for (int m = 0; m < rows; m++) v += lds[q / G_CH][m * G_CH + q % G_CH];
    if (d0 + q % G_CH < a.D) part[(long long)(q / G_CH) * a.D + q % G_CH] = v;
  }
}

// ddecay, dr_bias and di_bias from the tiles' partials [P][3][D], in 64 bits in a
// fixed order: 16 columns by 64 slices of the partials a block.
__global__ __launch_bounds__(1024) void k_gated_sums(const float *__restrict__ part, int P, int D, float *o0, float *o1,
                                                     float *o2) {
  __shared__ double sh[64][17];
  const int x = threadIdx.x & 15, y = threadIdx.x >> 4, k = blockIdx.y, d = (int)blockIdx.x * 16 + x;
  float *o = k == 0 ? o0 : k == 1 ? o1 : o2;
  if (!o) return;
  double s = 0;
  if (d < D)
    for (int p0 = y; p0 < P; p0 += 512) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; q++) v[q] = p0 + 64 * q < P ? part[((p0 + 64LL * q) * 3 + k) * D + d] : 0.f;
#pragma unroll
      for (int q = 0; q < 8; q++) s += (double)v[q];
    }
  sh[y][x] = s;
  for (int h = 32; h >= 1; h >>= 1) {
    __syncthreads();
    if (y < h) sh[y][x] += sh[y + h][x];
  }
  if (y == 0 && d < D) o[d] = (float)sh[0][x];
}

// ---------------------------------------------------------------------------
// one token
// ---------------------------------------------------------------------------
struct GatedStepArgs {
  const void *x, *r, *i;
  void *y;
  long long sx, sr, si, sy;
  const float *decay, *rb, *ib;
  float *state;
  const int *slots;
  int B, D, nslots;
};

// One token: four channels a thread.  64 x 2048 in bf16: 2.9 us, the latency of a
// launch, of the slot's load and of the row's behind it; a call takes 8.
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
    const VecU<float, V> h = ldu<float, V>(hp, n);
    const Consts4<T> cs = gated_consts<T>(a.decay, a.rb, a.ib, d, n);
#pragma unroll
    for (int k = 0; k < V; k++) {
      const GateVals g = gate_vals<T>(r.f(k), i.f(k), cs.c[k]);
      o[k] = decayed(g.a, GateConsts<T>::SHORT ? g.l * -LN2 : -g.l, h.f(k), g.m * g.i * x.f(k));
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
  if (p->D > (1 << 22)) return fail(PR_EUNSUPPORTED, "D = %d: at most 2^22", p->D);
  return PR_OK;
}

// Steps of a lane and wavefronts of a tile: forwards a lane keeps a and b of
// each step, back five values and two inputs.
struct GatedGeom {
  int k, nw;
};
GatedGeom gated_geom(int dtype, bool adj) {
  if (!adj) return dtype == PR_BF16 ? GatedGeom{8, 4} : GatedGeom{4, 4};
  return dtype == PR_BF16 ? GatedGeom{4, 4} : GatedGeom{2, 8};
}

struct GatedPlan {
  int waves, tt, tiles, cb;
  long long cols;
  size_t off_agg, off_sagg, off_spre, off_part, clear, bytes;
};
int gated_plan(const pr_gated_problem *p, bool adj, GatedPlan *pl) {
  const int rc = gated_check(p, false);
  if (rc != PR_OK) return rc;
  const GatedGeom g = gated_geom(p->dtype, adj);
  const int k4 = 4 * g.k;  // steps of a wavefront
  pl->waves = p->T >= g.nw * k4 ? g.nw : (p->T + k4 - 1) / k4;
  pl->tt = pl->waves * k4;
  pl->tiles = (p->T + pl->tt - 1) / pl->tt;
  pl->cb = (p->D + G_CH - 1) / G_CH;
  pl->cols = (long long)p->B * pl->cb;
  if ((double)pl->cols * pl->tiles * 64 > 1e12 || (double)p->B * pl->tiles >= 2147483648.0)
    return fail(PR_EUNSUPPORTED, "problem too large: %lld columns of %d tiles", pl->cols, pl->tiles);
  size_t o = 0;
  const size_t words = (size_t)pl->cols * 64 * 8, supers = (pl->tiles + G_SUPER - 1) / G_SUPER;
  if (pl->tiles > 1) {
    o = (size_t)pl->cols * 64;
    pl->off_agg = o; o += words * pl->tiles;
    pl->off_sagg = o; o += words * supers;
    pl->off_spre = o; o += words * supers;
  } else {
    pl->off_agg = pl->off_sagg = pl->off_spre = 0;
  }
  pl->clear = o;
  o = (o + 255) & ~(size_t)255;
  pl->off_part = o;
  if (adj) o += ((size_t)p->B * pl->tiles * 3 * p->D * 4 + 255) & ~(size_t)255;
  pl->bytes = o > 256 ? o : 256;
  return PR_OK;
}

// The chain in the workspace, marked as empty where there is one.
hipError_t gated_chain(const GatedPlan &pl, void *workspace, GatedChain *ch, hipStream_t s) {
  char *ws = (char *)workspace;
  ch->ticket = (unsigned *)ws;
  ch->agg = (unsigned long long *)(ws + pl.off_agg);
  ch->sagg = (unsigned long long *)(ws + pl.off_sagg);
  ch->spre = (unsigned long long *)(ws + pl.off_spre);
  ch->cols = pl.cols;
  if (!pl.clear) return hipSuccess;
  const long long n = (long long)(pl.clear / 16), blocks = (n + 255) / 256;
  k_gated_clear<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, s>>>((uint4 *)ws, n);
  return hipGetLastError();
}

// A tile's offsets in an array are 32-bit: at most 128 steps of 2^22 elements of 4 bytes.
int stride_ok(const View &v, int T) {
  if (v.p && T > 1 && (v.st < 0 || v.st > (1 << 22)))
    return fail(PR_EUNSUPPORTED, "time stride %lld: 0 to 2^22 elements", v.st);
  return PR_OK;
}

View view(const pr_view *v) { return v && v->p ? View{v->p, v->sb, v->st} : View{nullptr, 0, 0}; }

int gated_fill(const pr_gated_problem *p, const GatedPlan &pl, const pr_gated_inputs *in, GatedArgs *a) {
  if (!in) return fail(PR_EINVAL, "inputs are NULL");
  if (!in->x.p || !in->r.p || !in->i.p || !in->decay) return fail(PR_EINVAL, "x, r, i and decay are required");
  a->x = view(&in->x); a->r = view(&in->r); a->i = view(&in->i);
  for (const View *v : {&a->x, &a->r, &a->i}) {
    const int rc = stride_ok(*v, p->T);
    if (rc != PR_OK) return rc;
  }
  a->decay = in->decay; a->rb = in->r_bias; a->ib = in->i_bias; a->h0 = in->h0; a->lengths = in->lengths;
  a->B = p->B; a->T = p->T; a->D = p->D;
  a->cb = pl.cb; a->tiles = pl.tiles; a->tt = pl.tt;
  a->nst = (p->T + PR_GATED_STATE_STEPS - 1) / PR_GATED_STATE_STEPS;
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
  GatedPlan fw, ad;
  if (gated_plan(p, false, &fw) != PR_OK || gated_plan(p, true, &ad) != PR_OK) return 0;
  return with_adjoint && ad.bytes > fw.bytes ? ad.bytes : fw.bytes;
}

int pararnn_gated_scan(const pr_gated_problem *p, const pr_gated_inputs *in, const pr_view *y, float *h_last,
                       float *states, void *workspace, size_t ws_bytes, void *stream) {
  clear_error();
  GatedPlan pl;
  int rc = gated_plan(p, false, &pl);
  if (rc != PR_OK) return rc;
  GatedArgs a{};
  if ((rc = gated_fill(p, pl, in, &a)) != PR_OK) return rc;
  if (!y || !y->p) return fail(PR_EINVAL, "y is required");
  if ((rc = check_ws(workspace, ws_bytes, pl.bytes)) != PR_OK) return rc;
  a.y = view(y); a.hlast = h_last; a.states = states;
  if ((rc = stride_ok(a.y, p->T)) != PR_OK) return rc;
  hipStream_t s = (hipStream_t)stream;
  GatedChain ch;
  HIPCHK(gated_chain(pl, workspace, &ch, s));
  const dim3 grid = flat_grid(pl.cols * pl.tiles);
  if (p->dtype == PR_BF16) k_gated_fwd<uint16_t, 8, 4, 4><<<grid, 64 * pl.waves, 0, s>>>(a, ch);
  else k_gated_fwd<float, 4, 4, 4><<<grid, 64 * pl.waves, 0, s>>>(a, ch);
  HIPCHK(hipGetLastError());
  return PR_OK;
}

int pararnn_gated_adjoint(const pr_gated_problem *p, const pr_gated_inputs *in, const float *states, const pr_view *dy,
                          const float *dh_last, const pr_gated_grads *gr, void *workspace, size_t ws_bytes,
                          void *stream) {
  clear_error();
  GatedPlan pl;
  int rc = gated_plan(p, true, &pl);
  if (rc != PR_OK) return rc;
  GatedArgs a{};
  if ((rc = gated_fill(p, pl, in, &a)) != PR_OK) return rc;
  if (!states || !dy || !dy->p || !gr) return fail(PR_EINVAL, "states, dy and the gradients' struct are required");
  if ((rc = check_ws(workspace, ws_bytes, pl.bytes)) != PR_OK) return rc;
  a.y = view(dy); a.dx = view(&gr->x); a.dr = view(&gr->r); a.di = view(&gr->i);
  for (const View *v : {&a.y, &a.dx, &a.dr, &a.di})
    if ((rc = stride_ok(*v, p->T)) != PR_OK) return rc;
  a.states = (float *)states; a.dhlast = dh_last; a.dh0 = gr->h0; a.h0 = nullptr;
  const bool sums = gr->decay || gr->r_bias || gr->i_bias;
  char *ws = (char *)workspace;
  a.part = sums ? (float *)(ws + pl.off_part) : nullptr;
  hipStream_t s = (hipStream_t)stream;
  GatedChain ch;
  HIPCHK(gated_chain(pl, workspace, &ch, s));
  const dim3 grid = flat_grid(pl.cols * pl.tiles);
  if (p->dtype == PR_BF16) k_gated_adj<uint16_t, 4, 4, 3><<<grid, 64 * pl.waves, 0, s>>>(a, ch);
  else k_gated_adj<float, 2, 8, 4><<<grid, 64 * pl.waves, 0, s>>>(a, ch);
  HIPCHK(hipGetLastError());
  if (!sums) return PR_OK;
  k_gated_sums<<<dim3((unsigned)((p->D + 15) / 16), 3), 1024, 0, s>>>(a.part, p->B * pl.tiles, p->D, gr->decay,
                                                                      gr->r_bias, gr->i_bias);
  HIPCHK(hipGetLastError());
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
