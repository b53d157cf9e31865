// A whole sparse layer for a few tokens (up to 16) in two kernels.
//
//   l_t = x_t Wg^T;  (I_t, w_t) = route(l_t)
//   h_p = act(x_t Wup[e]^T)            for each pair p = (t, k), e = I_t[k]
//   y_t = sum_k w_tk h_p Wdown[e]^T  (+ the shared expert's, weight 1)
//   act: relu(u)^2, or silu(u_gate) u_up of two halves of the up rows
//
// Bound by HBM: each used expert's weights are read once, whatever the number
// of tokens that use it, and everything else is small; so what counts is that
// the weights' stream starts early and never pauses.  The first kernel computes
// the logits (64-bit sums, rounded once to fp32) and clears the second one's
// counters.  The second one's work-groups each route all tokens by themselves
// (a wave a token), list the used experts, and then draw items from one
// counter: first blocks of rows of the up projections, expert by expert, then
// blocks of the down projections.  A down item waits until its expert's hidden
// rows are written, all of which have lower numbers; a work-group that holds
// an up item never waits, so the item with the lowest number is always worked
// on, whichever work-groups run.  The pairs' output rows are added by the
// wave that finishes a block of columns last, in a fixed order: same bits every
// time.
//
// Weights are the MFMA's A operand, read from HBM as whole lines into
// registers two stages ahead (across items) and decoded exactly to bf16 (8-bit:
// the block's scale on its sum).  The tokens' operand is bf16, too: a value that
// is no bf16 number (fp32 x, the hidden rows) is taken as the sum of three, 24
// bits, so products are exact to fp32 and sums are fp32 sums; the extra matrix
// instructions run in the time that the weights take to arrive.
#include <type_traits>

#include "fp8_device.h"
#include "gemm_device.h"
#include "kernels.h"
#include "mxfp4_device.h"
#include "route_device.h"

namespace lmoe {

namespace {

constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kMaxPairs = 1024;    // T K
constexpr int kXBytes = 48 * 1024; // the tokens' operand in LDS

struct MoeParams {
  MoeTokens m;
  float *logits, *h, *hs, *o;
  int32_t *next, *up_done, *down_done;
};

// Formats: k values in a line of 128 bytes, row groups of 16 that an item
// holds, lines a wave loads at a time, fragments of 8 values in 16 bytes.
template <int FMT>
struct Fmt;
template <>
struct Fmt<0> {  // bf16
  static constexpr int LK = 64, RG = 1, U = 2, NF = 1;
};
template <>
struct Fmt<1> {  // MXFP4
  static constexpr int LK = 256, RG = 2, U = 1, NF = 4;
};
template <>
struct Fmt<2> {  // FP8
  static constexpr int LK = 128, RG = 2, U = 1, NF = 2;
};

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
  const u16x4 v = *reinterpret_cast<const u16x4*>(p);
  return f32x4{bf16_to_f32(v[0]), bf16_to_f32(v[1]), bf16_to_f32(v[2]), bf16_to_f32(v[3])};
}

}  // namespace

// Logits: a work-group an expert, products and sums in 64 bits.
template <class GT, class XT>
__global__ __launch_bounds__(256) void moe_logits_kernel(const XT* __restrict__ x, long x_stride,
                                                         const GT* __restrict__ gate, int T, int E,
                                                         int D, float* __restrict__ logits,
                                                         int32_t* __restrict__ sync, int nsync) {
  constexpr int TB = 8;
  __shared__ double part[4][TB];
  const int e = blockIdx.x, tid = threadIdx.x;
  if (e == 0)
    for (int i = tid; i < nsync; i += 256) sync[i] = 0;
  for (int t0 = 0; t0 < T; t0 += TB) {
    double acc[TB];
#pragma unroll
    for (int u = 0; u < TB; ++u) acc[u] = 0.0;
    for (int k = tid * 4; k < D; k += 1024) {
      const f32x4 g = load4(gate + (size_t)e * D + k);
#pragma unroll
      for (int u = 0; u < TB; ++u) {
        if (t0 + u >= T) break;
        const f32x4 v = load4(x + (t0 + u) * x_stride + k);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[u] = fma((double)g[i], (double)v[i], acc[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < TB; ++u) {
      if (t0 + u >= T) break;
      const double s = wave_sum(acc[u]);
      if ((tid & 63) == 0) part[tid >> 6][u] = s;
    }
    __syncthreads();
    if (tid < TB && t0 + tid < T)
      logits[(size_t)(t0 + tid) * E + e] =
          (float)(part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid]);
    __syncthreads();
  }
}

namespace {

// What a work-group works on: block `blk` of rows of expert slot u (-1: the
// shared expert) in one of the two projections.
struct Item {
  int valid, down, u, blk;
};

// One projection of one expert.
struct Matrix {
  const uint8_t* w;  // codes
  const uint8_t* s;  // scales
  int K, rows;       // rows: of one half where gated
};

}  // namespace

template <int FMT, int NJ>
__global__ __launch_bounds__(kThreads, 4) void moe_tokens_kernel(MoeParams p) {
  using C = Fmt<FMT>;
  constexpr int LK = C::LK, RG = C::RG, U = C::U, NF = C::NF;
  constexpr int LANES = kWaves * U;  // lines of a stage, over the waves
  constexpr int RW = NJ >= 16 ? 4 : 8;
  constexpr int RED = kWaves * RG * 64 * 16;
  constexpr int ROUTE = RW * (256 + NJ * 512);
  static_assert(ROUTE + kMaxPairs * 4 + 2 * 4096 <= kXBytes + RED, "prologue's room");
  __shared__ __attribute__((aligned(16))) char smem[kXBytes + RED];
  __shared__ float sw[kMaxPairs];               // pairs' weights
  __shared__ uint16_t slist[kMaxPairs];         // pairs by expert
  __shared__ uint16_t sexp[kMaxPairs], sstart[kMaxPairs + 1];  // used experts, their first pair
  __shared__ int stick, scount[kWaves];

  const MoeTokens& m = p.m;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = uniform(tid >> 6);
  const int T = m.T, E = m.r.E, K = m.r.K, D = m.D, F = m.F, S = m.S, gated = m.gated;
  const int P = T * K;

  // ---- routing and the list of used experts, in every work-group ----
  int first = 0;
  if (tid == 0) first = __hip_atomic_fetch_add(p.next, 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  int32_t* const sidx = reinterpret_cast<int32_t*>(smem + ROUTE);
  uint32_t* const smask = reinterpret_cast<uint32_t*>(smem + ROUTE + kMaxPairs * 4);
  uint32_t* const sfirst = smask + 1024;
  for (int i = tid; i < E; i += kThreads) smask[i] = 0;
  if (w < RW)
    for (int t = w; t < T; t += RW)
      route_token<float, NJ>(p.logits + (size_t)t * E, m.bias, m.r, lane,
                             reinterpret_cast<float*>(smem + w * 256),
                             smem + RW * 256 + w * NJ * 512, sidx + t * K, sw + t * K);
  __syncthreads();
  for (int i = tid; i < P; i += kThreads) {
    atomicOr(&smask[sidx[i]], 1u << (i / K));
    if (blockIdx.x == 0) {
      m.idx[i] = sidx[i];
      m.weights[i] = sw[i];
    }
  }
  __syncthreads();
  int nu;
  {
    // thread i: experts 2 i and 2 i + 1; low half: used experts, high half: pairs
    const uint32_t a = 2 * tid < E ? smask[2 * tid] : 0u;
    const uint32_t b = 2 * tid + 1 < E ? smask[2 * tid + 1] : 0u;
    const int va = a ? 1 | (__popc(a) << 16) : 0, vb = b ? 1 | (__popc(b) << 16) : 0;
    int inc = va + vb;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(inc, off, 64);
      if (lane >= off) inc += o;
    }
    if (lane == 63) scount[w] = inc;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      if (i < w) before += scount[i];
      total += scount[i];
    }
    nu = total & 0xFFFF;
    const int at = before + inc - va - vb;
    if (a) {
      sexp[at & 0xFFFF] = (uint16_t)(2 * tid);
      sstart[at & 0xFFFF] = (uint16_t)(at >> 16);
      sfirst[2 * tid] = at >> 16;
    }
    if (b) {
      sexp[(at + va) & 0xFFFF] = (uint16_t)(2 * tid + 1);
      sstart[(at + va) & 0xFFFF] = (uint16_t)((at + va) >> 16);
      sfirst[2 * tid + 1] = (at + va) >> 16;
    }
    if (tid == 0) {
      sstart[nu] = (uint16_t)P;
      stick = first;
    }
  }
  __syncthreads();
  for (int i = tid; i < P; i += kThreads) {
    const int e = sidx[i], t = i / K;
    slist[sfirst[e] + __popc(smask[e] & ((1u << t) - 1u))] = (uint16_t)i;
  }
  nu = uniform(nu);
  const int fr = 16 * RG >> gated;  // hidden columns of an up item
  const int nf = (F + fr - 1) / fr, ns = (S + fr - 1) / fr, nd = D / (16 * RG);
  const int nup = ns + nu * nf, nexp = nu + (S > 0), total = nup + nexp * nd;
  int cur = uniform(stick);
  int next = cur + 1;
  __syncthreads();  // (the lists; smem is free)

  auto item_of = [&](int i) __attribute__((always_inline)) {
    Item it;
    it.valid = i < total;
    it.down = i >= nup;
    if (i < ns) {
      it.u = -1;
      it.blk = i;
    } else if (i < nup) {
      it.u = (i - ns) / nf;
      it.blk = (i - ns) - it.u * nf;
    } else {
      const int j = i - nup;
      it.u = j / nd - (S > 0);
      it.blk = j - (j / nd) * nd;
    }
    return it;
  };
  auto matrix_of = [&](const Item& it) __attribute__((always_inline)) {
    Matrix x;
    const int hid = it.u < 0 ? S : F;
    x.K = it.down ? hid : D;
    x.rows = it.down ? D : hid;
    x.w = static_cast<const uint8_t*>(it.u < 0 ? (it.down ? m.sdown : m.sup)
                                               : (it.down ? m.down : m.up));
    x.s = static_cast<const uint8_t*>(it.u < 0 ? (it.down ? m.sdown_s : m.sup_s)
                                               : (it.down ? m.down_s : m.up_s));
    const size_t e = it.u < 0 ? 0 : uniform(sexp[it.u]);
    const size_t rows = (size_t)x.rows << (gated && !it.down);
    x.w += e * rows * (FMT == 0 ? x.K * 2 : FMT == 1 ? x.K / 2 : x.K);
    if (FMT == 1) x.s += e * rows * (x.K / 32);
    if (FMT == 2) x.s += e * (rows / 128) * (x.K / 128) * 4;
    return x;
  };
  // Row of the matrix that row r (0 .. 15) of group g of a block is: where
  // gated, rows 0 - 7 are of the gate's half, 8 - 15 the same of the other.
  auto row_of = [&](const Item& it, const Matrix& x, int g, int r) __attribute__((always_inline)) {
    if (gated && !it.down) return it.blk * 8 * RG + 8 * g + (r & 7) + (r >= 8 ? x.rows : 0);
    return it.blk * 16 * RG + 16 * g + r;
  };

  const int r16 = lane & 15, kq = lane >> 4;
  const int src0 = (((r16 & 7) << 3) | kq) * 4;
  const int src1 = (((r16 & 7) << 3) | (4 + kq)) * 4;
  const bool lo = r16 < 8;

  struct Stage {
    u32x4 l[U][RG][2];
    uint32_t s[U][FMT == 1 ? RG : 1][2];
  };
  auto lines_of = [&](int k) __attribute__((always_inline)) { return (k + LK - 1) / LK; };
  // Stage st: lines w + kWaves (st U + u) of the block's rows.  (MXFP4: where K
  // ends in half a line, its second half reads the first one's bytes again,
  // and x is 0 there.)
  auto load = [&](Stage& A, const Item& it, const Matrix& x, int st) __attribute__((always_inline)) {
    const int lines = lines_of(x.K);
    const uint32_t rb = FMT == 0 ? x.K * 2 : FMT == 1 ? x.K / 2 : x.K;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int l = w + kWaves * (st * U + u);
      if (l >= lines) break;
      const bool half = FMT == 1 && l * LK + LK > x.K;
      const uint32_t at = l * 128 + (half ? lane & 3 : lane & 7) * 16;
#pragma unroll
      for (int g = 0; g < RG; ++g) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          A.l[u][g][h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(
              x.w + (size_t)((uint32_t)row_of(it, x, g, 8 * h + (lane >> 3)) * rb + at)));
        if (FMT == 1) {
          const uint32_t* sp = reinterpret_cast<const uint32_t*>(x.s) +
                               (uint32_t)row_of(it, x, g, r16) * (uint32_t)(x.K / 128) + 2 * l;
          A.s[u][g][0] = sp[0];
          A.s[u][g][1] = sp[half ? 0 : 1];
        }
      }
      if (FMT == 2)  // (a block's groups lie in one block of scales)
        A.s[u][0][0] = reinterpret_cast<const uint32_t*>(
            x.s)[(uint32_t)(row_of(it, x, 0, 4 * kq) / 128) * (uint32_t)(x.K / 128) + l];
    }
  };

  f32x4 acc[RG];
  // Adds stage st to acc.  x0: the lane's place in LDS of the first value of the
  // tokens' rows there (line l0 on), PN parts `plane` bytes apart; `on` is false
  // for lanes whose token is not among them (multi: only then there are some).
  auto compute = [&](auto pn, const Stage& A, int K_, int st, int l0, const char* x0, int plane,
                     bool multi, bool on) __attribute__((always_inline)) {
    constexpr int PN = decltype(pn)::value;
    const int lines = lines_of(K_);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int l = w + kWaves * (st * U + u);
      if (l >= lines) break;
      u32x4 c[RG][2];
#pragma unroll
      for (int g = 0; g < RG; ++g)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int a = (int)A.l[u][g][0][d], b = (int)A.l[u][g][1][d];
          const int a0 = __builtin_amdgcn_ds_bpermute(src0, a);
          const int b0 = __builtin_amdgcn_ds_bpermute(src0, b);
          const int a1 = __builtin_amdgcn_ds_bpermute(src1, a);
          const int b1 = __builtin_amdgcn_ds_bpermute(src1, b);
          c[g][0][d] = lo ? a0 : b0;
          c[g][1][d] = lo ? a1 : b1;
        }
      f32x4 blk[RG];
#pragma unroll
      for (int g = 0; g < RG; ++g) blk[g] = FMT == 2 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[g];
      const char* xl = x0 + (l - l0) * LK * 2;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < NF; ++i) {
          bf16x8 xf[PN];
#pragma unroll
          for (int q = 0; q < PN; ++q) {
            xf[q] = *reinterpret_cast<const bf16x8*>(xl + q * plane + h * 64 * NF + i * 16);
            if (multi && !on) xf[q] = zero8();
          }
#pragma unroll
          for (int g = 0; g < RG; ++g) {
            bf16x8 wf;
            if (FMT == 0) {
              wf = __builtin_bit_cast(bf16x8, c[g][h]);
            } else if (FMT == 1) {
              wf = mx_decode8(c[g][h][i], mx_scale((A.s[u][g][h] >> (8 * kq)) & 255u));
            } else {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const auto v0 =
                    __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[g][h][2 * i + j], 1.f, false);
                const auto v1 =
                    __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[g][h][2 * i + j], 1.f, true);
                wf[4 * j] = v0[0], wf[4 * j + 1] = v0[1];
                wf[4 * j + 2] = v1[0], wf[4 * j + 3] = v1[1];
              }
            }
#pragma unroll
            for (int q = 0; q < PN; ++q) blk[g] = mfma_bf16(wf, xf[q], blk[g]);
          }
        }
#pragma unroll
      for (int g = 0; g < RG; ++g)
        acc[g] = FMT == 2 ? acc[g] + blk[g] * __uint_as_float(A.s[u][0][0]) : blk[g];
    }
  };

  // Rows r0 .. r0 + n - 1 of the item's tokens (x, or hidden rows), values k0 ..
  // k0 + kn - 1, into LDS as parts of bf16; zeros from K on.
  auto put_rows = [&](const Item& it, int K_, int r0, int n, int k0, int kn, int pitch, int plane,
                      int parts) __attribute__((always_inline)) {
    for (int r = 0; r < n; ++r) {
      const int pair = it.u < 0 ? r0 + r : slist[sstart[it.u] + r0 + r];
      const int t = it.u < 0 ? pair : pair / K;
      const float* hrow = it.u < 0 ? p.hs + (size_t)pair * S : p.h + (size_t)pair * F;
      for (int k = tid * 4; k < kn; k += kThreads * 4) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (k0 + k < K_) {
          if (it.down) v = load4(hrow + k0 + k);
          else if (m.x_bf16) v = load4(static_cast<const uint16_t*>(m.x) + t * m.x_stride + k0 + k);
          else v = load4(static_cast<const float*>(m.x) + t * m.x_stride + k0 + k);
        }
        char* const to = smem + r * pitch + k * 2;
        for (int q = 0; q < parts; ++q) {
          const u16x4 b = pack4_bf16(v);
          *reinterpret_cast<u16x4*>(to + q * plane) = b;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] -= bf16_to_f32(b[i]);
        }
      }
    }
  };

  f32x4* const red = reinterpret_cast<f32x4*>(smem + kXBytes);  // [kWaves][RG][64]
  Stage A, B;
  Item it = item_of(cur);
  Matrix x = it.valid ? matrix_of(it) : Matrix{};
  if (it.valid) load(A, it, x, 0);
  while (it.valid) {
    int pending = 0;
    if (tid == 0)
      pending = __hip_atomic_fetch_add(p.next, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const Item nit = item_of(next);
    const Matrix nx = nit.valid ? matrix_of(nit) : Matrix{};
    const int r0 = it.u < 0 ? 0 : uniform(sstart[it.u]);
    const int rows = it.u < 0 ? T : uniform(sstart[it.u + 1]) - r0;
    const int parts = !it.down && m.x_bf16 ? 1 : 3;
    const int lines = lines_of(x.K);
    const int stages = (lines + LANES - 1) / LANES;
    // stages whose rows fit LDS at a time; where not even one does, a stage's
    // rows take turns (the products of the others' columns are with zeros)
    const int per = LANES * LK * 2;
    int chunk = (kXBytes / (rows * parts) - 16) / per;
    int turn = rows;
    if (chunk < 1) {
      chunk = 1;
      turn = kXBytes / (parts * (per + 16));
    }
    chunk = min(chunk, stages);
    const bool multi = turn < rows;
    const int pitch = min(chunk * LANES, lines) * LK * 2 + 16, plane = turn * pitch;
#pragma unroll
    for (int g = 0; g < RG; ++g) acc[g] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto step = [&](const Stage& Cur, Stage& Nxt, int st) __attribute__((always_inline)) {
      const int in = st % chunk;
      for (int b = 0; b < rows; b += turn) {
        const int n = min(turn, rows - b);
        if (in == 0) {
          if (st == 0 && b == 0 && it.down) {
            // the expert's hidden rows, all of them
            if (tid == 0) {
              // (bounded, about ten seconds: should a counter ever be wrong, the
              // result is, too, but the kernel ends)
              const int want = RG * (it.u < 0 ? ns : nf);
              for (int n = 0; n < (1 << 23); ++n) {
                if (__hip_atomic_load(p.up_done + it.u + 1, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) >= want)
                  break;
                __builtin_amdgcn_s_sleep(1);
              }
            }
            __syncthreads();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
          } else {
            __syncthreads();  // what is there has been read
          }
          const int k0 = st * LANES * LK;
          put_rows(it, x.K, b, n, k0, min(chunk * LANES * LK, lines * LK - k0), pitch, plane,
                   parts);
          __syncthreads();
        }
        if (b == 0) {
          if (st + 1 < stages) load(Nxt, it, x, st + 1);
          else if (st == stages - 1 && (stages & 1) == 0 && nit.valid) load(Nxt, nit, nx, 0);
        }
        const bool on = r16 >= b && r16 < b + n;
        const char* const x0 = smem + (on ? r16 - b : 0) * pitch + kq * NF * 16;
        const int l0 = (st - in) * LANES;
        if (parts == 1)
          compute(std::integral_constant<int, 1>{}, Cur, x.K, st, l0, x0, plane, multi, on);
        else
          compute(std::integral_constant<int, 3>{}, Cur, x.K, st, l0, x0, plane, multi, on);
      }
    };
    for (int st = 0; st < stages; st += 2) {
      step(A, B, st);
      if (st + 1 < stages) step(B, A, st + 1);
    }
    // (an odd number of stages: A was the last one read)
    if ((stages & 1) && nit.valid) load(A, nit, nx, 0);

#pragma unroll
    for (int g = 0; g < RG; ++g) red[(w * RG + g) * 64 + lane] = acc[g];
    if (tid == 0) stick = pending;
    __syncthreads();
    if (w < RG) {
      const int g = w;
      f32x4 v = red[g * 64 + lane];
#pragma unroll
      for (int i = 1; i < kWaves; ++i) v += red[(i * RG + g) * 64 + lane];
      const bool live = r16 < rows;
      const int pair = it.u < 0 ? r16 : (live ? slist[r0 + r16] : 0);
      if (!it.down) {
        float* const hrow = it.u < 0 ? p.hs + (size_t)pair * S : p.h + (size_t)pair * F;
        f32x4 o;
        int col;
        if (gated) {
          f32x4 b;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            b[i] = __shfl_xor(v[i], 32, 64);
            o[i] = v[i] / (1.f + expf(-v[i])) * b[i];
          }
          col = it.blk * fr + 8 * g + 4 * kq;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = relu_sq(v[i]);
          col = it.blk * fr + 16 * g + 4 * kq;
        }
        if (live && (!gated || kq < 2)) *reinterpret_cast<f32x4*>(hrow + col) = o;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
        if (lane == 0)
          __hip_atomic_fetch_add(p.up_done + it.u + 1, 1, __ATOMIC_RELAXED,
                                 __HIP_MEMORY_SCOPE_AGENT);
      } else {
        const int block = it.blk * RG + g, n0 = block * 16;
        float* const orow = p.o + (size_t)(it.u < 0 ? P + pair : pair) * D + n0;
        if (live)
          *reinterpret_cast<f32x4*>(orow + 4 * kq) = v * (it.u < 0 ? 1.f : sw[pair]);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
        int before = 0;
        if (lane == 0)
          before = __hip_atomic_fetch_add(p.down_done + block, 1, __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT);
        if (uniform(before) == nexp - 1) {
          // all pairs' rows of these columns are there: add them, k ascending
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
          for (int t = kq; t < T; t += 4) {
            const float* at = p.o + n0 + r16;
            float s = 0.f;
            for (int k = 0; k < K; ++k) s += at[(size_t)(t * K + k) * D];
            if (S > 0) s += at[(size_t)(P + t) * D];
            const size_t to = (size_t)t * D + n0 + r16;
            if (m.y_bf16) static_cast<uint16_t*>(m.y)[to] = f32_to_bf16(s);
            else static_cast<float*>(m.y)[to] = s;
          }
        }
      }
    }
    cur = next;
    next = uniform(stick);
    it = nit;
    x = nx;
    __syncthreads();
  }
}

namespace {

struct Layout {
  size_t sync, logits, h, hs, o, total;
  int nsync;
};
Layout layout(const MoeTokens& m) {
  Layout l{};
  auto take = [&](size_t bytes) {
    const size_t at = l.total;
    l.total += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t pairs = (size_t)m.T * m.r.K;
  l.nsync = 64 + m.r.E + 1 + m.D / 16;
  l.sync = take((size_t)l.nsync * 4);
  l.logits = take((size_t)m.T * m.r.E * 4);
  l.h = take(pairs * m.F * 4);
  l.hs = take((size_t)m.T * m.S * 4);
  l.o = take((pairs + (m.S ? m.T : 0)) * m.D * 4);
  return l;
}

template <int FMT, int NJ>
void launch(const MoeParams& p, int grid, hipStream_t s) {
  moe_tokens_kernel<FMT, NJ><<<grid, kThreads, 0, s>>>(p);
}

}  // namespace

size_t moe_tokens_workspace(const MoeTokens& m) { return layout(m).total; }

hipError_t moe_tokens(const MoeTokens& m, void* workspace, hipStream_t s) {
  const Layout l = layout(m);
  char* const ws = static_cast<char*>(workspace);
  int32_t* const sync = reinterpret_cast<int32_t*>(ws + l.sync);
  MoeParams p{m,
              reinterpret_cast<float*>(ws + l.logits),
              reinterpret_cast<float*>(ws + l.h),
              reinterpret_cast<float*>(ws + l.hs),
              reinterpret_cast<float*>(ws + l.o),
              sync,
              sync + 64,
              sync + 64 + m.r.E + 1};
  auto logits = [&](auto g, auto x) {
    using GT = decltype(g);
    using XT = decltype(x);
    moe_logits_kernel<GT, XT><<<m.r.E, 256, 0, s>>>(
        static_cast<const XT*>(m.x), m.x_stride, static_cast<const GT*>(m.gate), m.T, m.r.E, m.D,
        p.logits, sync, l.nsync);
  };
  if (m.gate_bf16 && m.x_bf16) logits(uint16_t{}, uint16_t{});
  else if (m.gate_bf16) logits(uint16_t{}, float{});
  else if (m.x_bf16) logits(float{}, uint16_t{});
  else logits(float{}, float{});
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int grid = 512;
  auto go = [&](auto fmt) {
    constexpr int FMT = decltype(fmt)::value;
    if (m.r.E <= 128) launch<FMT, 2>(p, grid, s);
    else if (m.r.E <= 512) launch<FMT, 8>(p, grid, s);
    else launch<FMT, 16>(p, grid, s);
  };
  if (m.format == 0) go(std::integral_constant<int, 0>{});
  else if (m.format == 1) go(std::integral_constant<int, 1>{});
  else go(std::integral_constant<int, 2>{});
  return hipGetLastError();
}

}  // namespace lmoe
