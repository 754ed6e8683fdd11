// Product of 8-bit integers with a scale for each row of both operands:
//   out[m][n] = (sum_k a[m][k] w[n][k]) sa[m] sw[n] + bias[n]
// Sums are exact in 32-bit integers on the i8 matrix instructions, so K may be
// split over wavefronts and blocks without a change in the result.
//
// Few rows (M <= 64): bound by reading w once.  A block takes 16 columns, its
// 8 wavefronts slices of K; a lane streams 64 adjacent bytes of one row of w
// straight into the operand registers of v_mfma_i32_16x16x64_i8, the rows of
// a (from cache) likewise, and the wavefronts' sums meet in shared memory.
// More rows: tiles staged through shared memory, v_mfma_i32_32x32x32_i8.
// Measured (to bf16, calls one after another on the same operands, which the
// caches hold in part; in brackets after 1 GiB of other writes): 16 x 4096 x 2048
// 5 us (7.5; by tiles 10), 64 x 4096 x 4096 13 us (19; by tiles 13 as well);
// 8192 cubed 439 to 485 us on three machines, 2.3 to 2.5 POP/s; 16384 x 8192 x
// 2048 300 to 342 us (the library's product to 32-bit integers 291), and where it
// took 312, 359 with 128 tiles and 425 staged through registers; 5000 x 1111 x
// 1111, of any alignment, 27 us (34).
#include "direct_rows.h"
#include "pararnn.h"
#include "ssm.h"

namespace pr {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct Gemm8Args {
  const int8_t *a, *w;
  const float *sa, *sw;
  const void *bias;
  void *out;
  int *part;  // K splits: [splits][M][N]
  long long lda, ldw, ldo;
  int M, N, K, splits, kper;  // kper: bytes of K per split
};

struct __attribute__((packed)) Bytes16 {
  i32x4 v;
};
// 16 bytes of a row from k on, zeros from `ke` on.  AL: 16-byte aligned and
// ke a multiple of 16; else any alignment, and the row's last bytes come from
// its last 16, moved down (one by one only in a row of fewer).
template <bool AL>
__device__ inline i32x4 load16(const int8_t *row, int k, int ke, bool on) {
  i32x4 v = {0, 0, 0, 0};
  if (!on || k >= ke) return v;
  if constexpr (AL) return *reinterpret_cast<const i32x4 *>(row + k);
  if (k + 16 <= ke) return reinterpret_cast<const Bytes16 *>(row + k)->v;
  if (ke >= 16) {
    v = reinterpret_cast<const Bytes16 *>(row + ke - 16)->v;
    const int s = 8 * (k + 16 - ke);  // bits, 8..120
    unsigned long long lo = (unsigned)v[0] | ((unsigned long long)(unsigned)v[1] << 32);
    unsigned long long hi = (unsigned)v[2] | ((unsigned long long)(unsigned)v[3] << 32);
    lo = s >= 64 ? hi >> (s - 64) : (lo >> s) | (hi << (64 - s));
    hi = s >= 64 ? 0 : hi >> s;
    return i32x4{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
  }
#pragma unroll
  for (int i = 0; i < 15; i++)
    if (k + i < ke) v[i / 4] |= (int)((unsigned)(uint8_t)row[k + i] << (8 * (i % 4)));
  return v;
}

template <typename T>
__device__ inline float scaled(const Gemm8Args &g, int v, int m, int n) {
  return fmaf((float)v, g.sa[m] * g.sw[n], g.bias ? ldf((const T *)g.bias, n) : 0.f);
}

// ---------------------------------------------------------------------------
template <typename T, int MT, bool AL>
__global__ __launch_bounds__(512) void k_gemm8_rows(Gemm8Args g) {
  __shared__ i32x4 red[8][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const bool non = n0 + r < g.N;
  const int8_t *wr = g.w + (long long)(non ? n0 + r : 0) * g.ldw;
  const int8_t *ar[MT];
  bool mon[MT];
#pragma unroll
  for (int i = 0; i < MT; i++) {
    mon[i] = i * 16 + r < g.M;
    ar[i] = g.a + (long long)(mon[i] ? i * 16 + r : 0) * g.lda;
  }
  i32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; i++) acc[i] = i32x4{0, 0, 0, 0};
  // lane (r, q) takes bytes 64 q .. 64 q + 63 of each 256: the order of k
  // within a step is the same in both operands
  for (int k0 = wave * 256 + q * 64; k0 - q * 64 < g.K; k0 += 8 * 256) {
    i32x4 b[4], a[MT][4];
#pragma unroll
    for (int s = 0; s < 4; s++) b[s] = load16<AL>(wr, k0 + s * 16, g.K, non);
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
      for (int s = 0; s < 4; s++) a[i][s] = load16<AL>(ar[i], k0 + s * 16, g.K, mon[i]);
#pragma unroll
    for (int s = 0; s < 4; s++)
#pragma unroll
      for (int i = 0; i < MT; i++) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[s], a[i][s], acc[i], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < MT; i++) red[wave][i][lane] = acc[i];
  __syncthreads();
  // register v of a lane: column n0 + 4 (lane / 16) + v, row lane % 16 of a
  for (int e = threadIdx.x; e < MT * 64; e += 512) {
    const int i = e >> 6, l = e & 63, m = i * 16 + (l & 15);
    if (m >= g.M) continue;
    i32x4 s = red[0][i][l];
#pragma unroll
    for (int k = 1; k < 8; k++) s += red[k][i][l];
#pragma unroll
    for (int v = 0; v < 4; v++) {
      const int n = n0 + 4 * (l >> 4) + v;
      if (n < g.N) stf((T *)g.out + m * g.ldo, n, scaled<T>(g, s[v], m, n));
    }
  }
}

// ---------------------------------------------------------------------------
// What a wavefront does with its 32 FM x 32 FN sums, from row mr0 and column
// nc0 on: a lane holds row lane % 32 of each 32 x 32 tile and, per 4
// registers, 4 adjacent columns 8 (v / 4) + 4 (lane / 32) ..
// K splits leave them to k_gemm8_join.  Else scaled, 32 rows at a time, through
// `mine`, a part of the block's shared memory of 32 rows that no other
// wavefront uses any more: stored as they are, an instruction would touch 32
// rows with a few bytes each; read back by rows it stores whole 128-byte lines.
// 16-byte chunks are swizzled by the row.
template <typename T, int FM, int FN>
__device__ inline void g8_results(const Gemm8Args &g, i32x16 (*acc)[FM], int8_t *mine, int mr0, int nc0, int lane) {
  const int h = lane >> 5, r = lane & 31;
  if (g.splits > 1) {
#pragma unroll
    for (int i = 0; i < FM; i++) {
      const int m = mr0 + i * 32 + r;
      if (m >= g.M) continue;
#pragma unroll
      for (int j = 0; j < FN; j++)
#pragma unroll
        for (int v4 = 0; v4 < 4; v4++) {
          const int n = nc0 + j * 32 + 8 * v4 + 4 * h;
          int *o = g.part + ((long long)blockIdx.y * g.M + m) * g.N + n;
          if (n + 4 <= g.N && (g.N & 3) == 0)
            *reinterpret_cast<i32x4 *>(o) = i32x4{acc[j][i][4 * v4], acc[j][i][4 * v4 + 1], acc[j][i][4 * v4 + 2],
                                                  acc[j][i][4 * v4 + 3]};
          else
            for (int c = 0; c < 4 && n + c < g.N; c++) o[c] = acc[j][i][4 * v4 + c];
        }
    }
    return;
  }
  constexpr int E = sizeof(T), CPR = FN * 32 * E / 16;  // chunks per row
  const bool vec = (g.ldo * E) % 16 == 0 && ((uintptr_t)g.out & 15) == 0;
  float sw[FN][16], bias[FN][16];  // of the lane's columns, loaded once
#pragma unroll
  for (int j = 0; j < FN; j++)
#pragma unroll
    for (int v = 0; v < 16; v++) {
      const int n = nc0 + j * 32 + 8 * (v >> 2) + 4 * h + (v & 3);
      sw[j][v] = n < g.N ? g.sw[n] : 0.f;
      bias[j][v] = n < g.N && g.bias ? ldf((const T *)g.bias, n) : 0.f;
    }
#pragma unroll
  for (int i = 0; i < FM; i++) {
    const int mr = mr0 + i * 32;
    const float sa = mr + r < g.M ? g.sa[mr + r] : 0.f;
#pragma unroll
    for (int j = 0; j < FN; j++)
#pragma unroll
      for (int v4 = 0; v4 < 4; v4++) {
        float o[4];
#pragma unroll
        for (int c = 0; c < 4; c++)
          o[c] = fmaf((float)acc[j][i][4 * v4 + c], sa * sw[j][4 * v4 + c], bias[j][4 * v4 + c]);
        const int byte = (j * 32 + 8 * v4 + 4 * h) * E, ch = (byte >> 4) ^ (r & (CPR - 1));
        int8_t *q = mine + r * (CPR * 16) + ch * 16 + (byte & 15);
        if constexpr (E == 2) {
          uint2 u;
          u.x = (unsigned)f2bf(o[0]) | ((unsigned)f2bf(o[1]) << 16);
          u.y = (unsigned)f2bf(o[2]) | ((unsigned)f2bf(o[3]) << 16);
          *reinterpret_cast<uint2 *>(q) = u;
        } else {
          *reinterpret_cast<float4 *>(q) = make_float4(o[0], o[1], o[2], o[3]);
        }
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wavefront's own stores, read by its other lanes
    if (vec) {
#pragma unroll
      for (int q = 0; q < 32 * CPR / 64; q++) {
        const int e = q * 64 + lane, row = e / CPR, ch = e % CPR;
        const int n = nc0 + ch * (16 / E), m = mr + row;
        const uint4 v = *reinterpret_cast<const uint4 *>(mine + row * (CPR * 16) + ((ch ^ (row & (CPR - 1))) << 4));
        if (m < g.M && n < g.N) {
          T *p = (T *)g.out + m * g.ldo + n;
          if (n + 16 / E <= g.N) {
            *reinterpret_cast<uint4 *>(p) = v;
          } else {
            const T *x = reinterpret_cast<const T *>(&v);
#pragma unroll
            for (int c = 0; c < 16 / E; c++)
              if (n + c < g.N) p[c] = x[c];
          }
        }
      }
    } else {  // rows of any alignment: neighbouring lanes store neighbouring elements
      constexpr int NC = FN * 32, RP = 64 / NC > 0 ? 64 / NC : 1, CP = NC / 64 > 0 ? NC / 64 : 1;
#pragma unroll 8
      for (int q = 0; q < 32 / RP * CP; q++) {
        const int row = q / CP * RP + (NC < 64 ? lane / NC : 0), col = (q % CP) * 64 + lane % (NC < 64 ? NC : 64);
        const int ch = col * E >> 4, n = nc0 + col, m = mr + row;
        const T x = *reinterpret_cast<const T *>(mine + row * (CPR * 16) + ((ch ^ (row & (CPR - 1))) << 4) +
                                                 (col * E & 15));
        if (m < g.M && n < g.N) ((T *)g.out)[m * g.ldo + n] = x;
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// ---------------------------------------------------------------------------
// 128 x 128 tile, K step 128 bytes, 4 wavefronts of 64 x 64.  Chunk c (16
// bytes) of tile row r sits at slot c ^ (r / 2 % 8) of its 128-byte line, so
// that the 16 rows of a fragment read fall on all 64 banks.
constexpr int TB = 128;
__device__ inline int t8_off(int r, int c) { return r * TB + ((c ^ ((r >> 1) & 7)) << 4); }

template <typename T, bool AL>
__global__ __launch_bounds__(256) void k_gemm8_tile(Gemm8Args g) {
  __shared__ __attribute__((aligned(16))) int8_t sA[2][128 * TB], sB[2][128 * TB];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
  const int tiles_n = (g.N + 127) / 128;
  const int m0 = (int)(blockIdx.x / tiles_n) * 128, n0 = (int)(blockIdx.x % tiles_n) * 128;
  const int kb = blockIdx.y * g.kper, ke = g.K - kb < g.kper ? g.K : kb + g.kper;
  i32x4 va[4], vb[4];
  auto gload = [&](int k0) {
#pragma unroll
    for (int q = 0; q < 4; q++) {
      const int e = tid + q * 256, r = e >> 3, k = k0 + (e & 7) * 16;
      va[q] = load16<AL>(g.a + (long long)(m0 + r) * g.lda, k, ke, m0 + r < g.M);
      vb[q] = load16<AL>(g.w + (long long)(n0 + r) * g.ldw, k, ke, n0 + r < g.N);
    }
  };
  auto lstore = [&](int buf) {
#pragma unroll
    for (int q = 0; q < 4; q++) {
      const int e = tid + q * 256, r = e >> 3, c = e & 7;
      *reinterpret_cast<i32x4 *>(&sA[buf][t8_off(r, c)]) = va[q];
      *reinterpret_cast<i32x4 *>(&sB[buf][t8_off(r, c)]) = vb[q];
    }
  };
  i32x16 acc[2][2];
#pragma unroll
  for (int j = 0; j < 2; j++)
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[j][i][r] = 0;
  int buf = 0;
  gload(kb);
  lstore(0);
  __syncthreads();
  const int ar = wm * 64 + (lane & 31), br = wn * 64 + (lane & 31), h = lane >> 5;
  for (int k0 = kb; k0 < ke; k0 += TB) {
    const bool more = k0 + TB < ke;
    if (more) gload(k0 + TB);
#pragma unroll
    for (int s = 0; s < 4; s++) {
      i32x4 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        a[i] = *reinterpret_cast<const i32x4 *>(&sA[buf][t8_off(ar + i * 32, 2 * s + h)]);
        b[i] = *reinterpret_cast<const i32x4 *>(&sB[buf][t8_off(br + i * 32, 2 * s + h)]);
      }
#pragma unroll
      for (int j = 0; j < 2; j++)
#pragma unroll
        for (int i = 0; i < 2; i++)
          acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[j], a[i], acc[j][i], 0, 0, 0);
    }
    if (more) lstore(buf ^ 1);
    __syncthreads();
    buf ^= 1;
  }
  g8_results<T, 2, 2>(g, acc, &sA[0][0] + wave * (32 * 64 * (int)sizeof(T)), m0 + wm * 64, n0 + wn * 64, lane);
}

// ---------------------------------------------------------------------------
// The same product with operands that go straight from memory to shared
// memory: a 16-byte buffer load of lane l fills bytes 16 l .. 16 l + 15 of a
// 1 KB run (8 tile rows of 128 bytes), so staging takes no registers and no
// stores; the layout above is made by which chunk each lane fetches.  Two
// stages of one 128-byte K step, an array each, so that the compiler can tell
// the stage being filled from the one being read.  Loads past M, N or the
// split's K write zeros: their vector offset lies outside the resource.
// WM x WN wavefronts of 32 FM x 32 FN.
typedef __amdgpu_buffer_rsrc_t G8Rsrc;
typedef __attribute__((address_space(3))) void g8_lds_t;

// this wavefront's loads have landed and its reads are done, then all meet
__device__ inline void g8_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(7 << 4);  // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <typename T, int WM, int WN, int FM, int FN>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_gemm8_direct(Gemm8Args g) {
  constexpr int BM = WM * FM * 32, BN = WN * FN * 32, NW = WM * WN, QA = BM / 8 / NW, QB = BN / 8 / NW;
  static_assert(QA % 2 == 0 && QB % 2 == 0 && QA <= 4 && QB <= 4, "even numbers of loads, at most four");
  static_assert(NW * 32 * FN * 32 * (int)sizeof(T) <= (BM + BN) * TB, "the results fit a stage");
  __shared__ __attribute__((aligned(1024))) int8_t s0[(BM + BN) * TB], s1[(BM + BN) * TB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN, h = lane >> 5;
  // Blocks go to the 8 dies in turn: each die takes a contiguous run of tiles,
  // eight rows of tiles at a time, so that its cache holds both operands' strips.
  const int tiles_m = (g.M + BM - 1) / BM, tiles_n = (g.N + BN - 1) / BN, tiles = tiles_m * tiles_n;
  int id = blockIdx.x;
  if (tiles % 8 == 0) id = (id % 8) * (tiles / 8) + id / 8;
  const int width = 8 * tiles_n, fm = (id / width) * 8, gm = min(tiles_m - fm, 8);
  const int m0 = (fm + (id % width) % gm) * BM, n0 = ((id % width) / gm) * BN;
  const int kb = blockIdx.y * g.kper, ke = g.K - kb < g.kper ? g.K : kb + g.kper;
  const G8Rsrc ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(g.a + m0 * g.lda), 0,
                                                      (int)(min(BM, g.M - m0) * g.lda), 0x00020000);
  const G8Rsrc rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(g.w + n0 * g.ldw), 0,
                                                      (int)(min(BN, g.N - n0) * g.ldw), 0x00020000);
  // (a load's chunk takes two values per lane: its number is even or odd)
  const int ce = direct_chunk(0, lane), co = direct_chunk(1, lane);
  unsigned ao[4], bo[4];
#pragma unroll
  for (int q = 0; q < QA; q++) ao[q] = direct_offset(wave * QA + q, lane, g.M - m0, (unsigned)g.lda);
#pragma unroll
  for (int q = 0; q < QB; q++) bo[q] = direct_offset(wave * QB + q, lane, g.N - n0, (unsigned)g.ldw);
  auto dload = [&](int8_t *d, int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < QA; q++)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (g8_lds_t *)&d[(wave * QA + q) * 1024], 16,
                                               k0 + ((q & 1) ? co : ce) < ke ? ao[q] : DIRECT_OOB, k0, 0, 0);
#pragma unroll
    for (int q = 0; q < QB; q++)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (g8_lds_t *)&d[BM * TB + (wave * QB + q) * 1024], 16,
                                               k0 + ((q & 1) ? co : ce) < ke ? bo[q] : DIRECT_OOB, k0, 0, 0);
  };
  i32x16 acc[FN][FM];
#pragma unroll
  for (int j = 0; j < FN; j++)
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[j][i][r] = 0;
  const int ar = wm * FM * 32 + (lane & 31), br = wn * FN * 32 + (lane & 31);
  // the next step's loads are in flight during the whole step; the fragments
  // of the next 32 k are read while this 32's products run
  auto step = [&](const int8_t *cur, int8_t *nx, int k0) __attribute__((always_inline)) {
    if (k0 + TB < ke) dload(nx, k0 + TB);
    i32x4 a[2][FM], b[2][FN];
    auto frag = [&](int w, int s) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < FM; i++) a[w][i] = *reinterpret_cast<const i32x4 *>(cur + t8_off(ar + i * 32, 2 * s + h));
#pragma unroll
      for (int j = 0; j < FN; j++)
        b[w][j] = *reinterpret_cast<const i32x4 *>(cur + BM * TB + t8_off(br + j * 32, 2 * s + h));
    };
    frag(0, 0);
    __builtin_amdgcn_sched_group_barrier(0x020, QA + QB, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, FM + FN, 0);
#pragma unroll
    for (int s = 0; s < 4; s++) {
      if (s < 3) frag((s + 1) & 1, s + 1);
#pragma unroll
      for (int j = 0; j < FN; j++)
#pragma unroll
        for (int i = 0; i < FM; i++)
          acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[s & 1][j], a[s & 1][i], acc[j][i], 0, 0, 0);
      if (s < 3) {
        constexpr int PAIRS = FM + FN < FM * FN ? FM + FN : FM * FN;
#pragma unroll
        for (int r = 0; r < PAIRS; r++) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, FM * FN - PAIRS, 0);
      }
    }
    g8_sync();
  };
  dload(s0, kb);
  g8_sync();
  int k0 = kb;
  for (; k0 + TB < ke; k0 += 2 * TB) {
    step(s0, s1, k0);
    step(s1, s0, k0 + TB);
  }
  if (k0 < ke) step(s0, s1, k0);
  g8_results<T, FM, FN>(g, acc, s0 + wave * (32 * FN * 32 * (int)sizeof(T)), m0 + wm * FM * 32, n0 + wn * FN * 32, lane);
}

template <typename T>
__global__ void k_gemm8_join(Gemm8Args g) {
  const long long mn = (long long)g.M * g.N, i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= mn) return;
  int s = 0;
  for (int k = 0; k < g.splits; k++) s += g.part[k * mn + i];
  const int m = (int)(i / g.N), n = (int)(i % g.N);
  stf((T *)g.out + m * g.ldo, n, scaled<T>(g, s, m, n));
}

// Edge of the block tile: 256 where its tiles fill the CUs, else 128 (4096
// cubed, 256 tiles: 73 us, 85 with 128; 1024 x 4096 x 4096, 64 tiles: 43 us, 30
// with 128).
static int gemm8_tile(int M, int N) {
  return (long long)((M + 255) / 256) * ((N + 255) / 256) >= 192 ? 256 : 128;
}

template <typename T, bool AL>
hipError_t gemm8_go(const Gemm8Args &g, hipStream_t s) {
  if (g.M <= 64) {
    const dim3 grid((unsigned)((g.N + 15) / 16));
    if (g.M <= 16) k_gemm8_rows<T, 1, AL><<<grid, 512, 0, s>>>(g);
    else if (g.M <= 32) k_gemm8_rows<T, 2, AL><<<grid, 512, 0, s>>>(g);
    else k_gemm8_rows<T, 4, AL><<<grid, 512, 0, s>>>(g);
    return hipGetLastError();
  }
  const int tile = gemm8_tile(g.M, g.N);
  const dim3 grid((unsigned)((long long)((g.M + tile - 1) / tile) * ((g.N + tile - 1) / tile)), (unsigned)g.splits);
  // (the direct loads' offsets in a tile are 31-bit)
  const bool direct = AL && g.lda < (1 << 22) && g.ldw < (1 << 22);
  if (tile == 256 && direct) k_gemm8_direct<T, 2, 4, 4, 2><<<grid, 512, 0, s>>>(g);
  else if (tile == 256) {
    const dim3 small((unsigned)((long long)((g.M + 127) / 128) * ((g.N + 127) / 128)), (unsigned)g.splits);
    k_gemm8_tile<T, AL><<<small, 256, 0, s>>>(g);
  } else if (direct) k_gemm8_direct<T, 2, 2, 2, 2><<<grid, 256, 0, s>>>(g);
  else k_gemm8_tile<T, AL><<<grid, 256, 0, s>>>(g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.splits == 1) return e;
  const long long mn = (long long)g.M * g.N;
  k_gemm8_join<T><<<dim3((unsigned)((mn + 255) / 256)), 256, 0, s>>>(g);
  return hipGetLastError();
}

// Splits of K where the tiles alone leave CUs idle: enough blocks for one
// round of the device, at least four K steps each (128 x 4096 x 4096: 18.0 us,
// 20.2 unsplit; 301 x 1030 x 1000: 17.0 and 18.6).
static int gemm8_splits(int M, int N, int K, int *kper) {
  const long long tiles = (long long)((M + 127) / 128) * ((N + 127) / 128);
  const int steps = (K + TB - 1) / TB;
  int s = M <= 64 || gemm8_tile(M, N) == 256 ? 1 : (int)(256 / tiles);
  if (s > steps / 4) s = steps / 4;
  if (s < 1) s = 1;
  const int per = (steps + s - 1) / s;
  *kper = per * TB;
  return (steps + per - 1) / per;
}

}  // namespace pr

using namespace pr;

namespace {

#define HIPCHK(expr)                                                                        \
  do {                                                                                      \
    hipError_t e_ = (expr);                                                                 \
    if (e_ != hipSuccess) return fail(PR_EHIP, "%s: %s", #expr, hipGetErrorString(e_));     \
  } while (0)

int gemm8_check(int M, int N, int K) {
  if (M < 1 || N < 1 || K < 1) return fail(PR_EINVAL, "sizes must be >= 1 (M=%d N=%d K=%d)", M, N, K);
  if (K >= 131072) return fail(PR_EUNSUPPORTED, "K = %d: sums of 131072 products may pass 32 bits", K);
  if (M > (1 << 30) || N > (1 << 30)) return fail(PR_EUNSUPPORTED, "M = %d, N = %d: at most 2^30", M, N);
  // a launch has 2^32 threads at most: 512 for 16 columns, 256 for a tile
  const double blocks = M <= 64 ? (N + 15) / 16 * 2.0 : (double)((M + 127) / 128) * ((N + 127) / 128);
  if (blocks >= (1 << 24)) return fail(PR_EUNSUPPORTED, "problem too large: %d x %d results", M, N);
  return PR_OK;
}

}  // namespace

extern "C" {

size_t pararnn_gemm_i8_workspace_bytes(int M, int N, int K) {
  clear_error();
  if (gemm8_check(M, N, K) != PR_OK) return 0;
  int kper;
  const int s = gemm8_splits(M, N, K, &kper);
  const size_t need = s > 1 ? (size_t)s * M * N * 4 : 0;
  return need > 256 ? (need + 255) & ~(size_t)255 : 256;
}

int pararnn_gemm_i8(int dtype, int M, int N, int K, const signed char *a, long long lda, const float *sa,
                    const signed char *w, long long ldw, const float *sw, const void *bias, void *out, long long ldo,
                    void *workspace, size_t ws_bytes, void *stream) {
  clear_error();
  if (dtype != PR_F32 && dtype != PR_BF16) return fail(PR_EINVAL, "unknown dtype %d", dtype);
  const int rc = gemm8_check(M, N, K);
  if (rc != PR_OK) return rc;
  if (!a || !sa || !w || !sw || !out) return fail(PR_EINVAL, "a, sa, w, sw and out are required");
  // one row has no stride: whatever stands for it (1 where it was a column) is not looked at
  if (M == 1) { lda = (K + 15LL) & ~15LL; ldo = N; }
  if (N == 1) ldw = (K + 15LL) & ~15LL;
  if (lda < K || ldw < K || ldo < N)
    return fail(PR_EINVAL, "row strides %lld, %lld, %lld are below K = %d, K, N = %d", lda, ldw, ldo, K, N);
  const size_t need = pararnn_gemm_i8_workspace_bytes(M, N, K);
  if (!workspace || ws_bytes < need) return fail(PR_EWORKSPACE, "workspace %zu bytes < %zu", ws_bytes, need);
  if (((uintptr_t)workspace & 255) != 0) return fail(PR_EINVAL, "workspace must be 256-byte aligned");
  Gemm8Args g{};
  g.a = (const int8_t *)a; g.w = (const int8_t *)w; g.sa = sa; g.sw = sw; g.bias = bias; g.out = out;
  g.part = (int *)workspace; g.lda = lda; g.ldw = ldw; g.ldo = ldo; g.M = M; g.N = N; g.K = K;
  g.splits = gemm8_splits(M, N, K, &g.kper);
  const bool al = K % 16 == 0 && lda % 16 == 0 && ldw % 16 == 0 && (((uintptr_t)a | (uintptr_t)w) & 15) == 0;
  hipStream_t s = (hipStream_t)stream;
  if (dtype == PR_BF16) HIPCHK((al ? gemm8_go<uint16_t, true>(g, s) : gemm8_go<uint16_t, false>(g, s)));
  else HIPCHK((al ? gemm8_go<float, true>(g, s) : gemm8_go<float, false>(g, s)));
  return PR_OK;
}

}  // extern "C"
