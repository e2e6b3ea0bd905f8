// Pieces of the tile kernels whose stages go straight from memory to LDS: the loader, a stage's
// barrier, the order of a step, the order of the tiles.
#pragma once

#include "gemm_kernel.h"

namespace fp8ds {

// LDS byte offset of 16-byte chunk c of row r, for rows of RB bytes.  A fragment read
// serves 16 consecutive rows at a time from the 16 16-byte columns of LDS; the chunks are
// permuted by the row so that those 16 pieces lie in 16 columns (two rows of 128 bytes, or
// four of 64, share the columns).
template <int RB>
__device__ __forceinline__ int chunk_off(int r, int c) {
  if constexpr (RB == 128) return r * 128 + ((c ^ ((r >> 1) & 7)) << 4);
  else return r * 64 + ((c ^ ((r >> 2) & 3)) << 4);
}

__device__ __forceinline__ void load_to_lds16(__amdgpu_buffer_rsrc_t rsrc, uint8_t* lds, int voff,
                                              int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      rsrc, (void __attribute__((address_space(3)))*)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void load_to_lds4(__amdgpu_buffer_rsrc_t rsrc, uint8_t* lds, int voff,
                                             int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      rsrc, (void __attribute__((address_space(3)))*)lds, 4, voff, soff, 0, 0);
}
// An offset past every buffer: such a load gives zeros and does not reach memory.
constexpr int kNowhere = 0x40000000;

// This wave's share of the loads of one operand tile (ROWS rows of RB bytes a stage).
template <int ROWS, int RB, int NW>
struct TileLoader {
  static constexpr int kRowsPer = 1024 / RB;  // rows per load instruction of a wave
  static constexpr int kPerWave = ROWS / kRowsPer / NW;
  static_assert(RB != 128 || kPerWave % 2 == 0, "a wave's first rows start a group of 16");
  __amdgpu_buffer_rsrc_t rsrc;
  int ld, w, row_off, col;

  __device__ __forceinline__ TileLoader(const uint8_t* src, int64_t ld_, int64_t row0, int64_t rows,
                                        int64_t row_bytes, int tid) {
    const int lane = tid & 63;
    ld = (int)ld_;
    w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the lane's place in the 1 KB that an instruction fills, and the chunk that belongs there
    const int row = lane / (RB / 16), place = lane % (RB / 16);
    col = (RB == 128 ? place ^ (row >> 1) : place ^ (row >> 2)) * 16;
    row_off = row * ld;
    const int64_t left = rows - row0 < ROWS ? rows - row0 : ROWS;
    rsrc = byte_rsrc(src + row0 * ld_, (left - 1) * ld_ + row_bytes);
  }

  // Bytes [k0, k0 + RB) of every row; what lies at or past row_bytes reads as zeros, and
  // so do rows past the matrix.
  __device__ __forceinline__ void issue(int k0, int row_bytes, uint8_t* lds) const {
    // rows 8 .. 15 of every 16 rows of 128 bytes have the other half of the permutations
    const int even = k0 + col < row_bytes ? row_off + col : kNowhere;
    const int odd = k0 + (col ^ 64) < row_bytes ? row_off + (col ^ 64) : kNowhere;
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int seg = w * kPerWave + i;
      load_to_lds16(rsrc, lds + seg * 1024, RB == 128 && (i & 1) ? odd : even,
                    seg * kRowsPer * ld + k0);
    }
  }
};

// Barrier of a stage: every wave's reads of LDS are done, and all but its last N loads.
// (__syncthreads would wait for all loads.)  The fences order this thread's accesses for
// the compiler and wait for nothing.
template <int N>
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  // vmcnt N, lgkmcnt 0, expcnt unconstrained
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The order of a step: DS fragment reads and VM loads spread over its MF MFMAs, the reads
// over the first three quarters so that the last of them has arrived for the next step.
template <int MF, int DS, int VM, int I = 0>
__device__ __forceinline__ void interleave() {
  if constexpr (I < MF) {
    constexpr int kSpan = MF * 3 / 4;
    constexpr int d0 = I < kSpan ? DS * I / kSpan : DS, d1 = I + 1 < kSpan ? DS * (I + 1) / kSpan : DS;
    constexpr int v0 = VM * I / MF, v1 = VM * (I + 1) / MF;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                              // MFMA
    if constexpr (d1 > d0) __builtin_amdgcn_sched_group_barrier(0x100, d1 - d0, 0);  // LDS read
    if constexpr (v1 > v0) __builtin_amdgcn_sched_group_barrier(0x020, v1 - v0, 0);  // VMEM read
    interleave<MF, DS, VM, I + 1>();
  }
}

// Tile of workgroup wg.  XCD x = wg % 8 takes a contiguous share of the tiles, which are
// numbered down groups of ROWS tile rows, so that the tiles an XCD works on at a time are
// near a square: 4 x 8 of the 32 of 256 x 256 (8 x 4: 258 us instead of 254 at
// 8192 x 14336 x 4096, 172 instead of 168 at 16384 x 4096 x 4096; 2 x 16: 258 and 171),
// 8 x 8 of the 64 of 128 x 128 (4 x 16: 47 us instead of 44 at 1000 x 14336 x 4096).
template <int ROWS>
__device__ __forceinline__ void tile_of(int wg, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int total = tiles_m * tiles_n, x = wg & 7;
  const int i = total < 8 ? wg : x * (total >> 3) + min(x, total & 7) + (wg >> 3);
  const int first = i / (ROWS * tiles_n) * ROWS, rows = min(tiles_m - first, ROWS);
  const int j = i - first * tiles_n;
  tm = first + j % rows;
  tn = j / rows;
}

}  // namespace fp8ds
