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

// The same at any alignment of an element (one access where all V are there,
// which the hardware takes unaligned; the first n one by one where they are not).
template <int BYTES>
struct WordsOf;
template <>
struct WordsOf<32> { typedef unsigned type __attribute__((ext_vector_type(8))); };
template <>
struct WordsOf<16> { typedef unsigned type __attribute__((ext_vector_type(4))); };
template <>
struct WordsOf<8> { typedef unsigned type __attribute__((ext_vector_type(2))); };
template <>
struct WordsOf<4> { typedef unsigned type; };
template <typename T, int V>
struct __attribute__((packed, aligned(sizeof(T)))) Packed {
  typename WordsOf<sizeof(T) * V>::type v;
};
template <typename T, int V>
struct VecU {
  union {
    typename WordsOf<sizeof(T) * V>::type v;
    T e[V];
  };
  __device__ float f(int i) const { return ldf(e, i); }
};
template <typename T, int V>
__device__ inline VecU<T, V> ldu(const T *p, int n) {
  VecU<T, V> r;
#pragma unroll
  for (int i = 0; i < V; i++) r.e[i] = 0;
  if (n >= V) {
    r.v = reinterpret_cast<const Packed<T, V> *>(p)->v;
  } else {
#pragma unroll
    for (int i = 0; i < V - 1; i++)
      if (i < n) r.e[i] = p[i];
  }
  return r;
}
template <typename T, int V>
__device__ inline void stu(T *p, const float *f, int n) {
  VecU<T, V> r;
#pragma unroll
  for (int i = 0; i < V; i++) stf(r.e, i, f[i]);
  if (n >= V) {
    reinterpret_cast<Packed<T, V> *>(p)->v = r.v;
  } else {
#pragma unroll
    for (int i = 0; i < V - 1; i++)
      if (i < n) p[i] = r.e[i];
  }
}
// The same for outputs that the call does not read again: stored non-temporally, they
// leave the caches to its inputs (a block's norms and their gradients, 16384 x 2048 in
// bf16: 177 to 166 us; the gated scan's training, 2 x 2048 x 2048: 64 to 54 us).
template <typename T, int V>
__device__ inline void stu_nt(T *p, const float *f, int n) {
  VecU<T, V> r;
#pragma unroll
  for (int i = 0; i < V; i++) stf(r.e, i, f[i]);
  typedef typename WordsOf<sizeof(T) * V>::type W __attribute__((aligned(sizeof(T))));
  if (n >= V) {
    __builtin_nontemporal_store(r.v, reinterpret_cast<W *>(p));
  } else {
#pragma unroll
    for (int i = 0; i < V - 1; i++)
      if (i < n) p[i] = r.e[i];
  }
}

}  // namespace pr
