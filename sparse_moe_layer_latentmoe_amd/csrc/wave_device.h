// Reductions over the lanes of a wave, the wait for its LDS accesses, and vector
// types beside lmoe_device.h's.
#pragma once
#include "lmoe_device.h"

namespace lmoe {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// v combined (by op) over each 16 consecutive lanes, in all of them: four DPP
// moves (lane ^ 1, lane ^ 2, mirrored halves, mirrored row), no LDS crossbar.
template <class Op>
__device__ __forceinline__ float row16_reduce(float v, Op op) {
#define LMOE_DPP(CTRL) \
  __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true))
  v = op(v, LMOE_DPP(0xB1));
  v = op(v, LMOE_DPP(0x4E));
  v = op(v, LMOE_DPP(0x141));
  v = op(v, LMOE_DPP(0x140));
#undef LMOE_DPP
  return v;
}

// v combined over the wave, in every lane (all lanes active).
template <class Op>
__device__ __forceinline__ float wave_reduce(float v, Op op) {
  v = row16_reduce(v, op);
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16 * i));
  return op(op(r[0], r[1]), op(r[2], r[3]));
}
struct AddOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct MaxOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// s_waitcnt with only the LDS counter set, to 0: this wave's LDS writes are
// done (stage_barrier does not wait for them).
__device__ __forceinline__ void wait_lgkmcnt0() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

}  // namespace lmoe
