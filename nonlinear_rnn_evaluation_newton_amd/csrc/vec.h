// V adjacent elements of storage type T moved as one access (16 bytes where
// V > 1), for the row and channel kernels.
#pragma once

#include "common.h"

namespace pr {

// A grid of more blocks than one dimension takes (2^32 threads): rows of 2^20
// blocks.  The last row may hold blocks past the end, which return at once.
// (A block's number does not take the grid's size, a load at the start of the
// kernel.)
inline dim3 flat_grid(long long blocks) {
  const long long x = blocks < (1 << 20) ? blocks : 1 << 20;
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}
__device__ inline long long flat_block() { return ((long long)blockIdx.y << 20) + blockIdx.x; }

template <typename T, int V>
struct Vec;
template <>
struct Vec<uint16_t, 8> { typedef uint4 type; };
template <>
struct Vec<uint16_t, 4> { typedef uint2 type; };
template <>
struct Vec<float, 4> { typedef float4 type; };
template <>
struct Vec<uint16_t, 1> { typedef uint16_t type; };
template <>
struct Vec<float, 1> { typedef float type; };
template <>
struct Vec<int8_t, 8> { typedef uint2 type; };
template <>
struct Vec<int8_t, 4> { typedef unsigned type; };
template <>
struct Vec<int8_t, 1> { typedef int8_t type; };

template <typename T, int V>
struct VecOf {
  union {
    typename Vec<T, V>::type v;
    T e[V];
  };
  __device__ float f(int i) const { return ldf(e, i); }
};
template <typename T, int V>
__device__ inline VecOf<T, V> ldv(const T *p, bool in) {
  VecOf<T, V> r;
  if (in) {
    r.v = *reinterpret_cast<const typename Vec<T, V>::type *>(p);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) r.e[i] = 0;
  }
  return r;
}
template <typename T, int V>
__device__ inline void stv(T *p, const float *f) {
  VecOf<T, V> r;
#pragma unroll
  for (int i = 0; i < V; i++) stf(r.e, i, f[i]);
  *reinterpret_cast<typename Vec<T, V>::type *>(p) = r.v;
}

}  // namespace pr
