// Device-side pieces shared by the LDS-tiled GEMMs: waits and barriers around
// direct global -> LDS copies, the work order over XCDs, and output through
// LDS.
#pragma once
#include "lmoe_device.h"

namespace lmoe {

// s_waitcnt with only the vector-memory counter set to N (gfx9 encoding:
// vmcnt bits [3:0] and [15:14], expcnt and lgkmcnt left at their maximum).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Workgroup barrier without a memory fence: the direct-to-LDS loads are
// waited for explicitly (wait_vmcnt) so that later stages stay in flight.
// The signal fences keep the compiler from moving LDS accesses across it.
__device__ __forceinline__ void stage_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Output of one wave's block of 16 TM rows, written through LDS.  In the
// MFMA result layout lane (r, q) (r = lane % 16, q = lane / 16) of tile
// (g, t) holds columns 16 g + 4 q .. + 3 of row 16 t + r, so a direct store
// instruction writes 16 pieces of 32 bytes.  Here tiles G0 .. G0 + GN - 1
// are packed (p.pack4: the stored bits of four columns) into `reg`, the
// wave's own LDS region of 16 TM rows x 32 GN bytes (16-byte chunks XOR-
// swizzled by row), and read back as 16 contiguous bytes per lane, so that
// each store instruction (p.store8) writes whole 32 GN-byte row pieces.
// Rows from `rows` on are not stored; row i goes to slot m0 + i, columns
// from n0.  Only this wave touches `reg`, and a wave's LDS accesses stay in
// order, so no barrier is needed inside.  Measured on the prefill batch's
// expert GEMMs (bitwise equal): MXFP4 up projection 3.41 against 3.45-3.56
// ms with direct stores, down projection 3.18 against 3.30-3.33 ms.
template <int GN, int G0, int TN, int TM, class P>
__device__ __forceinline__ void staged_store(const P& p, char* reg, int lane,
                                             const f32x4 (&acc)[TN][TM], int m0, int rows, int n0) {
  constexpr int RB = GN * 32, CH = RB / 16, RPI = 64 / CH;
  static_assert(G0 + GN <= TN && (CH & (CH - 1)) == 0 && CH <= 64, "staged store");
  const int r16 = lane & 15, kq = lane >> 4;
#pragma unroll
  for (int g = 0; g < GN; ++g)
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      const int row = t * 16 + r16;
      const int chunk = 2 * g + (kq >> 1);
      *reinterpret_cast<u16x4*>(reg + row * RB + ((chunk ^ (row & (CH - 1))) << 4) +
                                (kq & 1) * 8) = p.pack4(acc[G0 + g][t]);
    }
  const int c = lane & (CH - 1);
#pragma unroll
  for (int j = 0; j < 16 * TM / RPI; ++j) {
    const int row = j * RPI + lane / CH;
    const u16x8 v = *reinterpret_cast<const u16x8*>(reg + row * RB + ((c ^ (row & (CH - 1))) << 4));
    if (row < rows) p.store8(m0 + row, n0 + c * 8, v);
  }
}

typedef __attribute__((address_space(3))) void lds_void;

// Work-item order.  Work-groups are dealt to the 8 XCDs round-robin by id,
// and each XCD has its own L2, so XCD x is given the contiguous chunk x of
// the work list: the work-groups resident on one XCD at a time are then
// neighbours in the list and share operand panels in that XCD's L2 while
// they walk k in step.  List order: for the grouped expert GEMMs, expert by
// expert, n block by n block, the expert's m tiles fastest (they share the
// weight panel); for dense GEMMs, groups of kDenseGroupM m tiles, m fastest
// (8: measured on the prefill batch's dense GEMMs, 1-3% faster than 4 and
// within noise of 16).
constexpr int kXcds = 8;
constexpr int kDenseGroupM = 8;

template <bool GROUPED>
__device__ __forceinline__ bool work_item(int nblocks, int mrows, int bm, const Tile* tiles,
                                          const int* ntiles, int& tm, int& nb) {
  const int mtiles = GROUPED ? *ntiles : (mrows + bm - 1) / bm;
  const int total = mtiles * nblocks;
  const int chunk = (total + kXcds - 1) / kXcds;
  const int local = blockIdx.x / kXcds;
  const int item = (blockIdx.x % kXcds) * chunk + local;
  if (local >= chunk || item >= total) return false;
  if (GROUPED) {
    const Tile t = tiles[item / nblocks];
    const int i = item - t.first * nblocks;
    nb = i / t.count;
    tm = t.first + i % t.count;
  } else {
    const int gsz = kDenseGroupM * nblocks;
    const int g = item / gsz;
    const int gm = min(kDenseGroupM, mtiles - g * kDenseGroupM);
    const int r = item - g * gsz;
    tm = g * kDenseGroupM + r % gm;
    nb = r / gm;
  }
  return true;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base) {
  // raw buffer over 2 GiB from `base`: offsets are checked against this
  // bound by the hardware (reads past it return 0)
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, 0x7FFFFFF0,
                                           0x00020000);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A barrier that is also a hard scheduling boundary: no LDS read of the
// stage may be hoisted above it (its data is not there yet) and no read of
// the previous stage sunk below it (other waves overwrite that buffer next).
__device__ __forceinline__ void stage_barrier_hard() {
  __builtin_amdgcn_sched_barrier(0);
  stage_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// work_item with the tile list's fields read into scalar registers.
template <bool GROUPED>
__device__ __forceinline__ bool work_item_uniform(int nblocks, int mrows, int bm,
                                                  const Tile* tiles, const int* ntiles, int& tm,
                                                  int& nb) {
  const int mtiles = GROUPED ? uniform(*ntiles) : (mrows + bm - 1) / bm;
  const int total = mtiles * nblocks;
  const int chunk = (total + kXcds - 1) / kXcds;
  const int local = blockIdx.x / kXcds;
  const int item = (blockIdx.x % kXcds) * chunk + local;
  if (local >= chunk || item >= total) return false;
  if (GROUPED) {
    const int first = uniform(tiles[item / nblocks].first);
    const int count = uniform(tiles[item / nblocks].count);
    const int i = item - first * nblocks;
    nb = i / count;
    tm = first + i % count;
  } else {
    const int gsz = kDenseGroupM * nblocks;
    const int g = item / gsz;
    const int gm = min(kDenseGroupM, mtiles - g * kDenseGroupM);
    const int r = item - g * gsz;
    tm = g * kDenseGroupM + r % gm;
    nb = r / gm;
  }
  return true;
}

}  // namespace lmoe
