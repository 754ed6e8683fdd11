// Offsets of the loads that go straight from memory to shared memory in the
// products' tile kernels.  Plain integer code, also compiled for the host.
//
// A tile row is one K step of 128 bytes, eight chunks of 16.  Load u of a tile
// covers rows 8 u .. 8 u + 7, lane l row 8 u + l / 8; chunk c of row r sits at
// slot c ^ (r / 2 % 8) of its line, so lane l fetches chunk
// (l % 8) ^ (4 (u % 2) + l / 16).
//
// The address is resource base + vector offset + scalar offset, and only the
// vector offset is sure to be part of the range check: whether the scalar one
// is, and what becomes of one that lies past the resource, is left open.  So
// the vector offset by itself decides: it holds the row, and lies outside every
// resource where the row is past the operand's end.  The scalar offset is the
// K step's first byte, below a row's stride.
#pragma once

#ifdef __HIPCC__
#define PR_HOST_DEVICE __host__ __device__
#else
#define PR_HOST_DEVICE
#endif

namespace pr {

constexpr unsigned DIRECT_OOB = 0x80000000u;  // outside every resource

// byte of the K step that lane `lane` fetches in load u
PR_HOST_DEVICE inline int direct_chunk(int u, int lane) { return ((lane & 7) ^ (((u & 1) << 2) | (lane >> 4))) * 16; }

// vector offset of that fetch in a tile of `rows` rows of the operand, `ld`
// bytes apart
PR_HOST_DEVICE inline unsigned direct_offset(int u, int lane, int rows, unsigned ld) {
  const int row = u * 8 + (lane >> 3);
  return row < rows ? (unsigned)row * ld + (unsigned)direct_chunk(u, lane) : DIRECT_OOB;
}

}  // namespace pr
