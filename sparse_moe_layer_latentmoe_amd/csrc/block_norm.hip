// The norms around a block, with the block's gate and the residual's scale,
// in one pass over the rows; and their gradients.
//
//   ry = 1 / sqrt(mean(y^2) + eps)      n  = post * y * ry   (n = y without post)
//   h' = alpha * h + g * n              the residual stream after the block
//   rh = 1 / sqrt(mean(h'^2) + eps)     x  = pre * h' * rh   the next block's input
//
// With G the gradient of h' (its own plus what comes back through x):
//   a  = pre * dx, hn = h' rh           G  = dh' + rh (a - hn mean(a hn))
//   dh = alpha G                        dalpha = sum_t G h
//   dg = G n (summed over what g is broadcast over)
//   b  = post g G, yn = y ry            dy = ry (b - yn mean(b yn))
//   dpost = sum_t g G yn                dpre = sum_t dx hn
//
// A work-group (or one wave, for narrow rows) keeps a row in registers, so each
// value is read once and written once; sums are fp32, the results round once.
// 4099 rows of 8192, fp32 stream, bf16 block, bf16 gate [T, D]: forward 99 us
// (470 MB, 4.7 TB/s), backward 152 us (739 MB, 4.9 TB/s) and 5.8 us for the
// column sums; a large copy reaches 4.8 TB/s.  32 rows forward: 5.1 us, a launch
// and two reductions.
//
// HBM bounds the forward at 4096 to 16384 columns (96 to 107 us for as many
// values) and the look-ahead backward below at 4096 to 8192 (141 to 152 us).
// Widths just past a step of the launch shapes leave threads idle (2112: 155 and
// 191 us; 576: 152 and 210; 1024: 103 and 163).  The backward's other forms do
// not fit the registers and are bound by the traffic of what the compiler
// spills (a thread, at 4099 x 8192 values): fp32 stream and block 136 to 180
// bytes, 278 us (bf16 stream, fp32 block 28 to 92: 155 us);
// rows wider than 8192 384 to 436 bytes, 408 us; 2049 to 8192 columns without
// wide loads (a width that is no multiple of 8, or arrays not 16-byte aligned)
// 1.2 KB, 1238 us, and the forward there, one value a load, 225 us.
//
// The backward computes h' again from h and y rather than reading it: dalpha
// needs h anyway.  Column sums: each of a fixed number of work-groups keeps
// the sums of its rows in registers and writes them once; a second kernel
// adds those in order (no atomics, the same bits every time).
#include <type_traits>

#include "gemm_device.h"
#include "kernels.h"
#include "wave_device.h"

namespace lmoe {

namespace {

// A per-column or per-row vector whose type is known at run time.
struct ParamVec {
  const void* p;
  int bf16;
};

// Eight values of one thread.  VEC: eight consecutive columns from c; else
// columns c, c + TPR, ..., each below D.
template <int TPR, bool VEC>
__device__ __forceinline__ void load8v(const float* p, int c, int D, float (&v)[8]) {
  if constexpr (VEC) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p + c);
    const f32x4 b = *reinterpret_cast<const f32x4*>(p + c + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i * TPR < D ? p[c + i * TPR] : 0.f;
  }
}
template <int TPR, bool VEC>
__device__ __forceinline__ void load8v(const uint16_t* p, int c, int D, float (&v)[8]) {
  if constexpr (VEC) {
    const u16x8 a = *reinterpret_cast<const u16x8*>(p + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = bf16_to_f32(a[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i * TPR < D ? bf16_to_f32(p[c + i * TPR]) : 0.f;
  }
}
template <int TPR, bool VEC>
__device__ __forceinline__ void load8v(ParamVec q, size_t row, int c, int D, float (&v)[8]) {
  if (q.bf16)
    load8v<TPR, VEC>(static_cast<const uint16_t*>(q.p) + row, c, D, v);
  else
    load8v<TPR, VEC>(static_cast<const float*>(q.p) + row, c, D, v);
}
template <int TPR, bool VEC>
__device__ __forceinline__ void store8v(float* p, int c, int D, const float (&v)[8]) {
  if constexpr (VEC) {
    *reinterpret_cast<f32x4*>(p + c) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(p + c + 4) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i * TPR < D) p[c + i * TPR] = v[i];
  }
}
template <int TPR, bool VEC>
__device__ __forceinline__ void store8v(uint16_t* p, int c, int D, const float (&v)[8]) {
  if constexpr (VEC) {
    // one instruction for two values; rounds as f32_to_bf16
    f32x8 a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = v[i];
    *reinterpret_cast<bf16x8*>(p + c) = __builtin_convertvector(a, bf16x8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i * TPR < D) p[c + i * TPR] = f32_to_bf16(v[i]);
  }
}
__device__ __forceinline__ void fill8(float (&v)[8], float x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x;
}

// Sums over the TPR threads of a row, the same in every thread.  Rows wider
// than a wave go through LDS: two buffers in turn, so one barrier a sum is
// enough (a buffer is written again only after a barrier that every thread
// reaches after reading it).
template <int TPR>
struct RowSum {
  f32x2* lds;  // [2][TPR / 64]
  int turn = 0;
  __device__ f32x2 operator()(float a, float b) {
    a = wave_reduce(a, AddOp{});
    b = wave_reduce(b, AddOp{});
    if constexpr (TPR > 64) {
      constexpr int NW = TPR / 64;
      f32x2* buf = lds + turn * NW;
      turn ^= 1;
      if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = f32x2{a, b};
      // LDS only: loads of the next row stay in flight
      wait_lgkmcnt0();
      stage_barrier();
      a = b = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const f32x2 q = buf[w];
        a += q[0];
        b += q[1];
      }
    }
    return f32x2{a, b};
  }
};

// The threads of a row: TPR of them, NC times eight values each; 64 threads
// to a row share a work-group of 256 with three other rows.
template <int TPR>
constexpr int rows_per_group() { return TPR == 64 ? 4 : 1; }

}  // namespace

struct BlockNormDev {
  const void* h;
  const void* y;  // null: 0
  long hs, ys;    // row strides
  ParamVec pre, post, alpha, gate;  // null: absent (post: no norm of y; alpha, gate: 1)
  int gate_kind;                    // 0 none, 1 per channel, 2 per token, 3 both
  int T, D;
  float eps;
};

template <class HT, class YT, int TPR, int NC, bool VEC>
__global__ __launch_bounds__(TPR* rows_per_group<TPR>()) void block_norm_kernel(
    BlockNormDev p, HT* __restrict__ h_out, YT* __restrict__ x, float* __restrict__ stats) {
  __shared__ f32x2 lds[2 * TPR / 64];
  RowSum<TPR> row_sum{lds};
  const int tid = threadIdx.x % TPR;
  const int t = blockIdx.x * rows_per_group<TPR>() + threadIdx.x / TPR;
  if (t >= p.T) return;
  const int D = p.D;
  const HT* h = static_cast<const HT*>(p.h) + (size_t)t * p.hs;
  const YT* y = p.y ? static_cast<const YT*>(p.y) + (size_t)t * p.ys : nullptr;
  auto col = [&](int i) { return VEC ? (i * TPR + tid) * 8 : i * 8 * TPR + tid; };

  float yv[NC][8], hv[NC][8], gv[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = col(i);
    fill8(yv[i], 0.f);
    fill8(hv[i], 0.f);
    fill8(gv[i], 1.f);
    if (c < D) {
      if (y) load8v<TPR, VEC>(y, c, D, yv[i]);
      load8v<TPR, VEC>(h, c, D, hv[i]);
      if (p.gate_kind == 3)
        load8v<TPR, VEC>(p.gate, (size_t)t * D, c, D, gv[i]);
      else if (p.gate_kind == 1)
        load8v<TPR, VEC>(p.gate, 0, c, D, gv[i]);
    }
  }
  float gt = 1.f;
  if (p.gate_kind == 2)
    gt = p.gate.bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.gate.p)[t])
                     : static_cast<const float*>(p.gate.p)[t];
  float ry = 1.f, rh = 1.f;
  if (p.post.p) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int v = 0; v < 8; ++v) ss = fmaf(yv[i][v], yv[i][v], ss);
    ry = 1.0f / sqrtf(row_sum(ss, 0.f)[0] / D + p.eps);
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = col(i);
    if (c >= D) continue;
    float a[8], w[8];
    fill8(a, 1.f);
    fill8(w, 1.f);
    if (p.alpha.p) load8v<TPR, VEC>(p.alpha, 0, c, D, a);
    if (p.post.p) load8v<TPR, VEC>(p.post, 0, c, D, w);
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const float n = w[v] * (yv[i][v] * ry);
      hv[i][v] = a[v] * hv[i][v] + (gv[i][v] * gt) * n;
      ss = fmaf(hv[i][v], hv[i][v], ss);
    }
    store8v<TPR, VEC>(h_out + (size_t)t * D, c, D, hv[i]);
  }
  if (x) {
    rh = 1.0f / sqrtf(row_sum(ss, 0.f)[0] / D + p.eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = col(i);
      if (c >= D) continue;
      float w[8];
      fill8(w, 1.f);
      if (p.pre.p) load8v<TPR, VEC>(p.pre, 0, c, D, w);
#pragma unroll
      for (int v = 0; v < 8; ++v) w[v] = w[v] * (hv[i][v] * rh);
      store8v<TPR, VEC>(x + (size_t)t * D, c, D, w);
    }
  }
  if (stats && tid == 0) {
    stats[2 * (size_t)t] = ry;
    stats[2 * (size_t)t + 1] = rh;
  }
}

struct BlockNormBackDev {
  const float* stats;
  const void* dh_out;  // null: 0
  const void* dx;      // null: no gradient through x
  void* dh;            // outputs; null: not wanted
  void* dy;
  void* dgate;         // gate kinds 2 and 3
  int dgate_bf16;
  // column sums: slot of each in the partial sums, or -1
  int s_post, s_pre, s_alpha, s_gate, nsums;
  float* part;         // [work-groups][nsums][D]
};

template <class HT, class YT, int TPR, int NC, bool VEC>
__global__ __launch_bounds__(TPR* rows_per_group<TPR>()) void block_norm_backward_kernel(
    BlockNormDev p, BlockNormBackDev q) {
  __shared__ f32x2 lds[2 * TPR / 64];
  RowSum<TPR> row_sum{lds};
  const int tid = threadIdx.x % TPR;
  const int group = blockIdx.x * rows_per_group<TPR>() + threadIdx.x / TPR;
  const int ngroups = gridDim.x * rows_per_group<TPR>();
  const int D = p.D;
  const float invd = 1.0f / D;
  auto col = [&](int i) { return VEC ? (i * TPR + tid) * 8 : i * 8 * TPR + tid; };

  float spost[NC][8], spre[NC][8], salpha[NC][8], sgate[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    fill8(spost[i], 0.f);
    fill8(spre[i], 0.f);
    fill8(salpha[i], 0.f);
    fill8(sgate[i], 0.f);
  }
  for (int t = group; t < p.T; t += ngroups) {
    const HT* h = static_cast<const HT*>(p.h) + (size_t)t * p.hs;
    const YT* y = p.y ? static_cast<const YT*>(p.y) + (size_t)t * p.ys : nullptr;
    const HT* dho = q.dh_out ? static_cast<const HT*>(q.dh_out) + (size_t)t * D : nullptr;
    const YT* dx = q.dx ? static_cast<const YT*>(q.dx) + (size_t)t * D : nullptr;
    float hv[NC][8], yv[NC][8], gv[NC][8], G[NC][8], dxv[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = col(i);
      fill8(hv[i], 0.f);
      fill8(yv[i], 0.f);
      fill8(gv[i], 1.f);
      fill8(G[i], 0.f);
      fill8(dxv[i], 0.f);
      if (c < D) {
        load8v<TPR, VEC>(h, c, D, hv[i]);
        if (y) load8v<TPR, VEC>(y, c, D, yv[i]);
        if (dho) load8v<TPR, VEC>(dho, c, D, G[i]);
        if (dx) load8v<TPR, VEC>(dx, c, D, dxv[i]);
        if (p.gate_kind == 3)
          load8v<TPR, VEC>(p.gate, (size_t)t * D, c, D, gv[i]);
        else if (p.gate_kind == 1)
          load8v<TPR, VEC>(p.gate, 0, c, D, gv[i]);
      }
    }
    const float ry = q.stats[2 * (size_t)t], rh = q.stats[2 * (size_t)t + 1];
    if (p.gate_kind == 2) {
      const float gt = p.gate.bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.gate.p)[t])
                                   : static_cast<const float*>(p.gate.p)[t];
#pragma unroll
      for (int i = 0; i < NC; ++i) fill8(gv[i], gt);
    }
    // yv becomes yn = y ry
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int v = 0; v < 8; ++v) yv[i][v] *= ry;
    if (dx) {
      float s1 = 0.f;
      float hn[NC][8];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = col(i);
        fill8(hn[i], 0.f);
        if (c >= D) continue;
        float a[8], w[8], pr[8];
        fill8(a, 1.f);
        fill8(w, 1.f);
        fill8(pr, 1.f);
        if (p.alpha.p) load8v<TPR, VEC>(p.alpha, 0, c, D, a);
        if (p.post.p) load8v<TPR, VEC>(p.post, 0, c, D, w);
        if (p.pre.p) load8v<TPR, VEC>(p.pre, 0, c, D, pr);
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          hn[i][v] = (a[v] * hv[i][v] + gv[i][v] * (w[v] * yv[i][v])) * rh;
          spre[i][v] = fmaf(dxv[i][v], hn[i][v], spre[i][v]);
          dxv[i][v] *= pr[v];
          s1 = fmaf(dxv[i][v], hn[i][v], s1);
        }
      }
      const float m1 = row_sum(s1, 0.f)[0] * invd;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int v = 0; v < 8; ++v) G[i][v] += rh * (dxv[i][v] - hn[i][v] * m1);
    }
    // dh, the column sums, dg; dxv becomes b = post g G
    float s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = col(i);
      if (c >= D) {
        fill8(dxv[i], 0.f);
        continue;
      }
      float a[8], w[8], o[8];
      fill8(a, 1.f);
      fill8(w, 1.f);
      if (p.alpha.p) load8v<TPR, VEC>(p.alpha, 0, c, D, a);
      if (p.post.p) load8v<TPR, VEC>(p.post, 0, c, D, w);
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        salpha[i][v] = fmaf(G[i][v], hv[i][v], salpha[i][v]);
        const float dn = G[i][v] * gv[i][v];
        const float dg = G[i][v] * (w[v] * yv[i][v]);
        spost[i][v] = fmaf(dn, yv[i][v], spost[i][v]);
        sgate[i][v] += dg;
        s3 += dg;
        gv[i][v] = dg;
        dxv[i][v] = w[v] * dn;
        s2 = fmaf(dxv[i][v], yv[i][v], s2);
        o[v] = a[v] * G[i][v];
      }
      if (q.dh) store8v<TPR, VEC>(static_cast<HT*>(q.dh) + (size_t)t * D, c, D, o);
      if (p.gate_kind == 3 && q.dgate) {
        if (q.dgate_bf16)
          store8v<TPR, VEC>(static_cast<uint16_t*>(q.dgate) + (size_t)t * D, c, D, gv[i]);
        else
          store8v<TPR, VEC>(static_cast<float*>(q.dgate) + (size_t)t * D, c, D, gv[i]);
      }
    }
    if ((p.post.p && q.dy) || (p.gate_kind == 2 && q.dgate)) {
      const f32x2 s = row_sum(s2, s3);
      s2 = p.post.p ? s[0] * invd : 0.f;
      if (p.gate_kind == 2 && q.dgate && tid == 0) {
        if (q.dgate_bf16)
          static_cast<uint16_t*>(q.dgate)[t] = f32_to_bf16(s[1]);
        else
          static_cast<float*>(q.dgate)[t] = s[1];
      }
    }
    if (q.dy) {
      const float m2 = p.post.p ? s2 : 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = col(i);
        if (c >= D) continue;
#pragma unroll
        for (int v = 0; v < 8; ++v) dxv[i][v] = ry * (dxv[i][v] - yv[i][v] * m2);
        store8v<TPR, VEC>(static_cast<YT*>(q.dy) + (size_t)t * D, c, D, dxv[i]);
      }
    }
  }
  float* part = q.part + (size_t)group * q.nsums * D;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = col(i);
    if (c >= D) continue;
    if (q.s_post >= 0) store8v<TPR, VEC>(part + (size_t)q.s_post * D, c, D, spost[i]);
    if (q.s_pre >= 0) store8v<TPR, VEC>(part + (size_t)q.s_pre * D, c, D, spre[i]);
    if (q.s_alpha >= 0) store8v<TPR, VEC>(part + (size_t)q.s_alpha * D, c, D, salpha[i]);
    if (q.s_gate >= 0) store8v<TPR, VEC>(part + (size_t)q.s_gate * D, c, D, sgate[i]);
  }
}

// The training step's usual case (y, dh_out, dx, dh and dy all there, wide
// loads, rows up to 8192): the next row's loads are issued before the current
// row is worked on (a row of 8192 is 115 KB a CU, enough to cover HBM's
// latency; the general kernel above, which does not, took 220 us for the case
// at the top against 152), and the [D] parameters lie in LDS (1 where absent).  Registers
// are what limits it: the sums take 64 of a thread's 256 and each of the two
// rows up to 72, so a row stays as it was loaded and is converted again in
// each of its passes.  GATE: 0 a gate of [D], [T] or none, 1 [T, D] in bf16, 2
// [T, D] in fp32.
namespace {

// Eight values as they lie in memory.  renew() hides from the compiler that a
// later conversion gives the same values as an earlier one, so that it
// converts again instead of keeping them in registers in between.
template <class T>
struct Raw8;
template <>
struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const void* p, size_t i) {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
    a = q[0];
    b = q[1];
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = a[i], o[4 + i] = b[i];
  }
  __device__ __forceinline__ void renew() { asm volatile("" : "+v"(a), "+v"(b)); }
};
template <>
struct Raw8<uint16_t> {
  u16x8 a;
  __device__ __forceinline__ void load(const void* p, size_t i) {
    a = *reinterpret_cast<const u16x8*>(static_cast<const uint16_t*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = bf16_to_f32(a[i]);
  }
  __device__ __forceinline__ void renew() { asm volatile("" : "+v"(a)); }
};

}  // namespace

template <class HT, class YT, int TPR, int NC, int GATE>
__global__ __launch_bounds__(TPR* rows_per_group<TPR>()) void block_norm_backward_ahead_kernel(
    BlockNormDev p, BlockNormBackDev q) {
  using GT = typename std::conditional<GATE == 2, float, uint16_t>::type;
  __shared__ f32x2 lds[2 * TPR / 64];
  extern __shared__ __attribute__((aligned(16))) float par[];  // [4][D] alpha, post, pre, gate
  RowSum<TPR> row_sum{lds};
  const int tid = threadIdx.x % TPR;
  const int group = blockIdx.x * rows_per_group<TPR>() + threadIdx.x / TPR;
  const int ngroups = gridDim.x * rows_per_group<TPR>();
  const int D = p.D;
  const float invd = 1.0f / D;
  const bool post = p.post.p != nullptr;
  auto col = [&](int i) { return (i * TPR + tid) * 8; };
  for (int c = threadIdx.x; c < D; c += TPR * rows_per_group<TPR>())
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ParamVec w = i == 0 ? p.alpha : (i == 1 ? p.post : (i == 2 ? p.pre : p.gate));
      float v = 1.f;
      if (w.p && (i < 3 || p.gate_kind == 1))
        v = w.bf16 ? bf16_to_f32(static_cast<const uint16_t*>(w.p)[c])
                   : static_cast<const float*>(w.p)[c];
      par[i * D + c] = v;
    }
  __syncthreads();
  auto param = [&](int i, int c, float (&v)[8]) __attribute__((always_inline)) {
    load8v<TPR, true>(par + i * D, c, D, v);
  };

  float spost[NC][8], spre[NC][8], salpha[NC][8], sgate[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    fill8(spost[i], 0.f);
    fill8(spre[i], 0.f);
    fill8(salpha[i], 0.f);
    fill8(sgate[i], 0.f);
  }
  struct Row {
    Raw8<HT> h[NC], dho[NC];
    Raw8<YT> y[NC], dx[NC];
    Raw8<GT> g[GATE ? NC : 1];
    f32x2 st;
    float gt;
  };
  auto load_row = [&](Row& r, int t) __attribute__((always_inline)) {
    const size_t at = (size_t)t * D;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      // threads past the row's end read its first columns (used nowhere)
      const int c = col(i) < D ? col(i) : 0;
      r.h[i].load(p.h, (size_t)t * p.hs + c);
      r.y[i].load(p.y, (size_t)t * p.ys + c);
      r.dho[i].load(q.dh_out, at + c);
      r.dx[i].load(q.dx, at + c);
      if constexpr (GATE > 0) r.g[i].load(p.gate.p, at + c);
    }
    r.st = *reinterpret_cast<const f32x2*>(q.stats + 2 * (size_t)t);
    r.gt = 1.f;
    if (p.gate_kind == 2)
      r.gt = p.gate.bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p.gate.p)[t])
                         : static_cast<const float*>(p.gate.p)[t];
  };
  Row next;
  if (group < p.T) load_row(next, group);
  for (int t = group; t < p.T; t += ngroups) {
    Row row = next;
    if (t + ngroups < p.T) load_row(next, t + ngroups);
    const float ry = row.st[0], rh = row.st[1];
    // the values that two passes share: alpha h, g and n = post yn; yn = y ry
    auto gate = [&](int i, int c, float (&g)[8]) __attribute__((always_inline)) {
      if constexpr (GATE > 0) {
        row.g[i].get(g);
      } else {
        param(3, c, g);
#pragma unroll
        for (int v = 0; v < 8; ++v) g[v] *= row.gt;
      }
    };
    auto normed = [&](int i, float (&yn)[8]) __attribute__((always_inline)) {
      row.y[i].get(yn);
#pragma unroll
      for (int v = 0; v < 8; ++v) yn[v] *= ry;
    };
    auto renew = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        row.h[i].renew();
        row.dho[i].renew();
        row.y[i].renew();
        row.dx[i].renew();
        if constexpr (GATE > 0) row.g[i].renew();
      }
    };
    float s1 = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = col(i);
      if (c < D) {
        float h[8], yn[8], g[8], d[8], al[8], w[8], pr[8];
        row.h[i].get(h);
        row.dx[i].get(d);
        normed(i, yn);
        gate(i, c, g);
        param(0, c, al);
        param(1, c, w);
        param(2, c, pr);
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const float hn = (al[v] * h[v] + g[v] * (w[v] * yn[v])) * rh;
          spre[i][v] = fmaf(d[v], hn, spre[i][v]);
          s1 = fmaf(d[v] * pr[v], hn, s1);
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // one piece's values at a time
    }
    const float m1 = row_sum(s1, 0.f)[0] * invd;
    renew();
    // G, dh, the column sums, dg and b = post g G
    float s2 = 0.f, s3 = 0.f;
    float b[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = col(i);
      fill8(b[i], 0.f);
      if (c < D) {
        float h[8], yn[8], g[8], al[8], w[8], G[8], d[8], pr[8];
        row.h[i].get(h);
        normed(i, yn);
        gate(i, c, g);
        param(0, c, al);
        param(1, c, w);
        row.dho[i].get(G);
        row.dx[i].get(d);
        param(2, c, pr);
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          const float n = w[v] * yn[v];
          const float hn = (al[v] * h[v] + g[v] * n) * rh;
          G[v] += rh * (d[v] * pr[v] - hn * m1);
          salpha[i][v] = fmaf(G[v], h[v], salpha[i][v]);
          const float dn = G[v] * g[v];
          const float dg = G[v] * n;
          spost[i][v] = fmaf(dn, yn[v], spost[i][v]);
          if constexpr (GATE == 0) {
            sgate[i][v] += dg;
            s3 += dg;
          }
          g[v] = dg;
          b[i][v] = w[v] * dn;
          s2 = fmaf(b[i][v], yn[v], s2);
          G[v] *= al[v];
        }
        store8v<TPR, true>(static_cast<HT*>(q.dh) + (size_t)t * D, c, D, G);
        if constexpr (GATE > 0)
          if (q.dgate) store8v<TPR, true>(static_cast<GT*>(q.dgate) + (size_t)t * D, c, D, g);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    const f32x2 s = row_sum(s2, s3);
    const float m2 = post ? s[0] * invd : 0.f;
    if (p.gate_kind == 2 && q.dgate && tid == 0) {
      if (q.dgate_bf16)
        static_cast<uint16_t*>(q.dgate)[t] = f32_to_bf16(s[1]);
      else
        static_cast<float*>(q.dgate)[t] = s[1];
    }
    renew();
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = col(i);
      if (c >= D) continue;
      float yn[8];
      normed(i, yn);
#pragma unroll
      for (int v = 0; v < 8; ++v) b[i][v] = ry * (b[i][v] - yn[v] * m2);
      store8v<TPR, true>(static_cast<YT*>(q.dy) + (size_t)t * D, c, D, b[i]);
    }
  }
  float* part = q.part + (size_t)group * q.nsums * D;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = col(i);
    if (c >= D) continue;
    if (q.s_post >= 0) store8v<TPR, true>(part + (size_t)q.s_post * D, c, D, spost[i]);
    if (q.s_pre >= 0) store8v<TPR, true>(part + (size_t)q.s_pre * D, c, D, spre[i]);
    if (q.s_alpha >= 0) store8v<TPR, true>(part + (size_t)q.s_alpha * D, c, D, salpha[i]);
    if (q.s_gate >= 0) store8v<TPR, true>(part + (size_t)q.s_gate * D, c, D, sgate[i]);
  }
}

// Column sums: out[slot][c] = sum over g of part[g][slot][c], g in a fixed
// order.  A work-group adds 64 columns of one slot, its 16 waves every 16th
// group each.
struct ColumnOut {
  void* p[4];
  int bf16[4];
};
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ part,
                                                          int ngroups, int nsums, int D,
                                                          ColumnOut out) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane, slot = blockIdx.y;
  const size_t step = (size_t)nsums * D;
  float s = 0.f;
  if (c < D)
    for (int g0 = w; g0 < ngroups; g0 += 16 * 8) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = g0 + 16 * i < ngroups ? part[(g0 + 16 * i) * step + (size_t)slot * D + c] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < D) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += red[i][lane];
    if (out.bf16[slot])
      static_cast<uint16_t*>(out.p[slot])[c] = f32_to_bf16(s);
    else
      static_cast<float*>(out.p[slot])[c] = s;
  }
}

namespace {

bool vec_ok(const void* p, long stride, int bf16) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride % (bf16 ? 8 : 4) == 0;
}

// Rows that the backward's launch gives partial sums: enough work-groups to
// fill the GPU, and no more than there are rows.
int backward_tpr(int D) { return D <= 512 ? 64 : (D <= 2048 ? 256 : (D <= 8192 ? 512 : 1024)); }
int backward_blocks(int T, int D) {
  const int tpr = backward_tpr(D);
  const int rpg = tpr == 64 ? 4 : 1;
  const int want = tpr >= 512 ? 256 : 1024;
  const int need = (T + rpg - 1) / rpg;
  return need < want ? need : want;
}

template <class F>
void with_types(bool h_bf16, bool y_bf16, F f) {
  if (h_bf16 && y_bf16) f(uint16_t{}, uint16_t{});
  else if (h_bf16) f(uint16_t{}, float{});
  else if (y_bf16) f(float{}, uint16_t{});
  else f(float{}, float{});
}

BlockNormDev device_args(const BlockNormProblem& b) {
  return {b.h, b.y, b.h_stride, b.y_stride,
          {b.pre.p, b.pre.bf16}, {b.post.p, b.post.bf16}, {b.alpha.p, b.alpha.bf16},
          {b.gate.p, b.gate.bf16}, b.gate_kind, b.T, b.D, b.eps};
}

bool inputs_vec(const BlockNormProblem& b) {
  bool v = b.D % 8 == 0 && vec_ok(b.h, b.h_stride, b.h_bf16) &&
           (!b.y || vec_ok(b.y, b.y_stride, b.y_bf16));
  for (const NormParam* q : {&b.pre, &b.post, &b.alpha}) v = v && vec_ok(q->p, 0, 1);
  return v && (b.gate_kind == 2 || vec_ok(b.gate.p, 0, 1));
}

}  // namespace

int block_norm_max_width() { return 16384; }

hipError_t block_norm(const BlockNormProblem& b, void* h_out, void* x, float* stats,
                      hipStream_t s) {
  const BlockNormDev p = device_args(b);
  const bool vec = inputs_vec(b) && vec_ok(h_out, 0, 1) && vec_ok(x, 0, 1);
  with_types(b.h_bf16, b.y_bf16, [&](auto ht, auto yt) {
    using HT = decltype(ht);
    using YT = decltype(yt);
    auto launch = [&](auto tpr, auto nc) {
      constexpr int TPR = decltype(tpr)::value, NC = decltype(nc)::value;
      constexpr int RPG = rows_per_group<TPR>();
      const int grid = (b.T + RPG - 1) / RPG;
      if (vec)
        block_norm_kernel<HT, YT, TPR, NC, true><<<grid, TPR * RPG, 0, s>>>(
            p, static_cast<HT*>(h_out), static_cast<YT*>(x), stats);
      else
        block_norm_kernel<HT, YT, TPR, NC, false><<<grid, TPR * RPG, 0, s>>>(
            p, static_cast<HT*>(h_out), static_cast<YT*>(x), stats);
    };
    using std::integral_constant;
    if (b.D <= 512) launch(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (b.D <= 2048) launch(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (b.D <= 8192) launch(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
    else launch(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  });
  return hipGetLastError();
}

size_t block_norm_backward_part(int T, int D, int nsums) {
  const int rpg = backward_tpr(D) == 64 ? 4 : 1;
  return (size_t)backward_blocks(T, D) * rpg * nsums * D * sizeof(float);
}

hipError_t block_norm_backward(const BlockNormProblem& b, const BlockNormGrads& g, float* part,
                               hipStream_t s) {
  const BlockNormDev p = device_args(b);
  BlockNormBackDev q{};
  q.stats = g.stats;
  q.dh_out = g.dh_out;
  q.dx = g.dx;
  q.dh = g.dh;
  q.dy = g.dy;
  q.part = part;
  ColumnOut out{};
  int n = 0;
  auto slot = [&](void* to, int bf16) {
    if (!to) return -1;
    out.p[n] = to;
    out.bf16[n] = bf16;
    return n++;
  };
  q.s_post = slot(g.dpost, b.post.bf16);
  q.s_pre = slot(g.dpre, b.pre.bf16);
  q.s_alpha = slot(g.dalpha, b.alpha.bf16);
  q.s_gate = b.gate_kind == 1 ? slot(g.dgate, b.gate.bf16) : -1;
  q.nsums = n;
  q.dgate = b.gate_kind >= 2 ? g.dgate : nullptr;
  q.dgate_bf16 = b.gate.bf16;
  const bool vec = inputs_vec(b) && vec_ok(g.dh_out, 0, 1) && vec_ok(g.dx, 0, 1) &&
                   vec_ok(g.dh, 0, 1) && vec_ok(g.dy, 0, 1) &&
                   (b.gate_kind != 3 || vec_ok(g.dgate, 0, 1));
  const bool ahead = vec && b.y && g.dh_out && g.dx && g.dh && g.dy;
  const int grid = backward_blocks(b.T, b.D);
  // no rows: the column sums below are of nothing and write zeros
  if (b.T > 0) with_types(b.h_bf16, b.y_bf16, [&](auto ht, auto yt) {
    using HT = decltype(ht);
    using YT = decltype(yt);
    auto launch = [&](auto tpr, auto nc) {
      constexpr int TPR = decltype(tpr)::value, NC = decltype(nc)::value;
      constexpr int RPG = rows_per_group<TPR>();
      if constexpr (TPR < 1024)
        if (ahead) {
          const size_t lds = (size_t)4 * b.D * sizeof(float);
          if (b.gate_kind != 3)
            block_norm_backward_ahead_kernel<HT, YT, TPR, NC, 0><<<grid, TPR * RPG, lds, s>>>(p, q);
          else if (b.gate.bf16)
            block_norm_backward_ahead_kernel<HT, YT, TPR, NC, 1><<<grid, TPR * RPG, lds, s>>>(p, q);
          else
            block_norm_backward_ahead_kernel<HT, YT, TPR, NC, 2><<<grid, TPR * RPG, lds, s>>>(p, q);
          return;
        }
      if (vec)
        block_norm_backward_kernel<HT, YT, TPR, NC, true><<<grid, TPR * RPG, 0, s>>>(p, q);
      else
        block_norm_backward_kernel<HT, YT, TPR, NC, false><<<grid, TPR * RPG, 0, s>>>(p, q);
    };
    using std::integral_constant;
    if (b.D <= 512) launch(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (b.D <= 2048) launch(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (b.D <= 8192) launch(integral_constant<int, 512>{}, integral_constant<int, 2>{});
    else launch(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || n == 0) return e;
  const int rpg = backward_tpr(b.D) == 64 ? 4 : 1;
  column_sum_kernel<<<dim3((b.D + 63) / 64, n), 1024, 0, s>>>(part, grid * rpg, n, b.D, out);
  return hipGetLastError();
}

}  // namespace lmoe
