// Matrices in 8-bit floating point (e4m3, OCP: largest finite value 448) with
// an fp32 scale for each block of 128 along k, and their products.
//
//   activations x [M, K]: scale xs[m][k / 128]; weights w [N, K]: scale
//   ws[n / 128][k / 128].  value = code * scale.
//   y[m][n] = sum over blocks b of xs[m][b] ws[n / 128][b] (sum of codes' products)
//
// Each block's sum of code products is one MFMA 16x16x128 from a zero
// accumulator; it is scaled in fp32 into the running sum (four fused
// multiply-adds per MFMA and lane, which run beside the next MFMA).  That
// instruction cuts products far below the largest of their eight (see
// fp8_device.h): on ordinary values well below what a result rounded to bf16 or
// e4m3 keeps, with a few large values among small ones about as much.  It is
// taken only where its rate is the bound (tiles) and the result is bf16 or
// e4m3.  fp32 results, and bf16 ones where weights are streamed, take the bf16
// MFMA on converted codes (EXACT: four 16x16x32, sums in fp32).  Weights
// are the MFMA's A operand and tokens its B operand, so a lane's four results
// are consecutive columns of one token and the scale is one factor per lane.
//
// A fragment is 32 bytes of a row; which k a lane holds does not matter as
// long as both operands agree, so lane (r, q) (r = lane % 16, q = lane / 16)
// takes the 16-byte chunks q and 4 + q of row r's 128 bytes.
#include <type_traits>

#include "fp8_copies.h"
#include "fp8_device.h"
#include "gemm_device.h"
#include "kernels.h"
#include "wave_device.h"

namespace lmoe {

namespace {

// ---- quantisation ------------------------------------------------------------

// A block's scale: largest magnitude / 448, at least the smallest normal
// number (a block of zeros, or of numbers below 448 of those).
__device__ __forceinline__ float fp8_scale(float amax) {
  return fmaxf(amax / kE4M3Max, 0x1p-126f);
}

// x / s, correctly rounded: r = 1 / s correctly rounded, then one Markstein
// correction of x r (exact residual by a fused multiply-add), three
// operations instead of a division.  The residual must not underflow, so
// very small scales take the division itself.  For x = -0 the residual is +0
// and the sum +0: where x may be -0, the sign is x's (s > 0).
__device__ __forceinline__ float fp8_ratio(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}
constexpr float kFastScale = 0x1p-90f;

// Eight values / s as e4m3 codes (round to nearest, ties to even).
__device__ __forceinline__ u32x2 fp8_pack8(const float (&v)[8], float s) {
  float q[8];
  if (s >= kFastScale) {
    const float r = 1.0f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = copysignf(fp8_ratio(v[i], s, r), v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] / s;
  }
  return u32x2{fp8_pack4(q[0], q[1], q[2], q[3]), fp8_pack4(q[4], q[5], q[6], q[7])};
}

// Eight values of a row from column c; columns from `cols` on read as 0.
template <bool VEC>
__device__ __forceinline__ void fp8_load8(const uint16_t* p, int c, int cols, float (&v)[8]) {
  if (VEC && c + 8 <= cols) {
    const u16x8 a = *reinterpret_cast<const u16x8*>(p + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = bf16_to_f32(a[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? bf16_to_f32(p[c + i]) : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void fp8_load8(const float* p, int c, int cols, float (&v)[8]) {
  if (VEC && c + 8 <= cols) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p + c);
    const f32x4 b = *reinterpret_cast<const f32x4*>(p + c + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? p[c + i] : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void fp8_store8(uint8_t* p, int c, int cols, u32x2 q) {
  if (VEC && c + 8 <= cols) {
    *reinterpret_cast<u32x2*>(p + c) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) p[c + i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
  }
}

__device__ __forceinline__ float max8(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

}  // namespace

// Activations: 16 lanes to a block of 128 values, each block on its own.
// Bound by HBM: 8192 x 8192 bf16 34 us (6.0 TB/s; two bytes read to one
// written), 192 x 10240 3.3 us.
template <class T, bool VEC>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(const T* __restrict__ x, long rows,
                                                           int cols, long stride, int nb,
                                                           uint8_t* __restrict__ codes,
                                                           float* __restrict__ scales) {
  const long blocks = rows * nb;
  const long b = (long)blockIdx.x * 16 + threadIdx.x / 16;
  if (b >= blocks) return;  // whole groups of 16 lanes
  const long row = b / nb;
  const int c = (int)(b - row * nb) * 128 + (threadIdx.x & 15) * 8;
  float v[8];
  fp8_load8<VEC>(x + row * stride, c, cols, v);
  const float s = fp8_scale(row16_reduce(max8(v), MaxOp{}));
  fp8_store8<VEC>(codes + row * cols, c, cols, fp8_pack8(v, s));
  if ((threadIdx.x & 15) == 0) scales[b] = s;
}

// Weights: a work-group to a block of 128 x 128; 16 lanes to a row piece,
// 16 rows at a time.
template <class T, bool VEC>
__global__ __launch_bounds__(256) void fp8_quantize_weight_kernel(const T* __restrict__ w, int rows,
                                                                  int cols, int rb, int cb,
                                                                  uint8_t* __restrict__ codes,
                                                                  float* __restrict__ scales) {
  __shared__ float wm[4];
  const int kb = blockIdx.x % cb;
  const long q = blockIdx.x / cb;
  const int nb = (int)(q % rb);
  const long base = q / rb * rows;  // first row of the matrix
  const int c = kb * 128 + (threadIdx.x & 15) * 8;
  const int r0 = nb * 128 + threadIdx.x / 16;
  float v[8][8];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    if (r < rows) {
      fp8_load8<VEC>(w + (base + r) * cols, c, cols, v[i]);
      m = fmaxf(m, max8(v[i]));
    }
  }
  m = wave_reduce(m, MaxOp{});
  if ((threadIdx.x & 63) == 0) wm[threadIdx.x >> 6] = m;
  __syncthreads();
  const float s = fp8_scale(fmaxf(fmaxf(wm[0], wm[1]), fmaxf(wm[2], wm[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    if (r < rows) fp8_store8<VEC>(codes + (base + r) * cols, c, cols, fp8_pack8(v[i], s));
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

// ---- tile list of a grouped product -------------------------------------------

// Tiles of at most tile_m rows of each group, from its row ranges offsets[g]
// .. offsets[g + 1] - 1, cut to [0, rows) and to rows that come after each
// other; one work-group, thread g for group g.
__global__ __launch_bounds__(1024) void fp8_tiles_kernel(const int32_t* __restrict__ offsets, int G,
                                                         int rows, int tile_m, int max_tiles,
                                                         Tile* __restrict__ tiles,
                                                         int32_t* __restrict__ ntiles) {
  __shared__ int part[16];
  const int g = threadIdx.x, lane = g & 63, w = g >> 6;
  int beg = 0, n = 0;
  if (g < G) {
    beg = min(max(offsets[g], 0), rows);
    n = max(min(max(offsets[g + 1], 0), rows) - beg, 0);
  }
  const int nt = (n + tile_m - 1) / tile_m;
  int inc = nt;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(inc, off, 64);
    if (lane >= off) inc += o;
  }
  if (lane == 63) part[w] = inc;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (i < w) before += part[i];
    total += part[i];
  }
  const int first = before + inc - nt;
  // offsets that do not ascend could ask for more tiles than rows allow:
  // such groups are dropped whole, so that no tile points past the list
  if (first + nt <= max_tiles)
    for (int i = 0; i < nt; ++i)
      tiles[first + i] = Tile{g, beg + i * tile_m, min(tile_m, n - i * tile_m), first, nt, 0, 0, 0};
  if (total <= max_tiles) {
    if (g == 0) *ntiles = total;
  } else if (first <= max_tiles && first + nt > max_tiles) {
    *ntiles = first;  // one group: those after it start past the list
  }
}

// ---- products -------------------------------------------------------------------

namespace {

// Row of x that row m of the product reads, and whether there is one (a row
// index outside x reads row 0 with a scale of 0).
__device__ __forceinline__ long fp8_x_row(const Fp8Gemm& p, int m, bool& ok) {
  ok = true;
  if (!p.rows) return m;
  const int r = p.rows[m];
  ok = r >= 0 && r < p.x_rows;
  return ok ? r : 0;
}

// What a product stores: float or uint16_t (bf16) rows of y, or the
// activation relu(v)^2 quantised again (codes in y, a scale for each 128
// columns in ys; N a multiple of 128).
struct Relu2Fp8 {};

// A fragment as the products take it.
template <bool EXACT>
using Frag = typename std::conditional<EXACT, Bf16Frag, i32x8>::type;
template <bool EXACT>
__device__ __forceinline__ Frag<EXACT> as_frag(i32x8 a) {
  if constexpr (EXACT) return fp8_to_bf16(a);
  else return a;
}

// Four values (squares: no -0 among them) / s as codes.
__device__ __forceinline__ uint32_t fp8_codes4(f32x4 v, float s) {
  if (s >= kFastScale) {
    const float r = 1.0f / s;
    return fp8_pack4(fp8_ratio(v[0], s, r), fp8_ratio(v[1], s, r), fp8_ratio(v[2], s, r),
                     fp8_ratio(v[3], s, r));
  }
  return fp8_pack4(v[0] / s, v[1] / s, v[2] / s, v[3] / s);
}

template <class OUT>
__device__ __forceinline__ void fp8_store4(const Fp8Gemm& p, int m, int n, f32x4 v) {
  OUT* y = static_cast<OUT*>(p.y) + (size_t)m * p.N + n;
  if constexpr (std::is_same<OUT, float>::value)
    *reinterpret_cast<f32x4*>(y) = v;
  else if constexpr (std::is_same<OUT, uint16_t>::value)
    store4_bf16(y, v);
}

// Fragment of rows 0-15 from the two 8-row loads a (rows 0-7) and b: lane
// (r, q) takes 16-byte chunk c of row r, held by lane 8 (r % 8) + c.
__device__ __forceinline__ i32x4 fp8_permute(const i32x4& a, const i32x4& b, int src4, bool lo) {
  i32x4 r;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int va = __builtin_amdgcn_ds_bpermute(src4, a[d]);
    const int vb = __builtin_amdgcn_ds_bpermute(src4, b[d]);
    r[d] = lo ? va : vb;
  }
  return r;
}

}  // namespace

// Few tokens: every weight byte is read once, as whole cache lines, and k is
// split over the NW waves of a work-group, whose sums are added in LDS in a
// fixed order.  A wave instruction loads 8 rows x 128 bytes; ds_bpermute
// moves the pieces to the MFMA's lanes (the layout that the bf16 streaming
// GEMM measured fastest).  Work-group: 16 RG weight rows x 16 token rows.
// Bound by HBM: 1 x 10240 x 8192 15.5 us (5.4 TB/s; 14.8 with the 8-bit
// instruction's sums), 32 tokens' 704 rows over 512 experts 577 to 591 us at
// 5120 x 2048 (6.9 to 7.0 TB/s; 583 to 588).
template <bool GROUPED, int NW, int RG, int U, class OUT>
__global__ __launch_bounds__(NW * 64) void fp8_stream_kernel(Fp8Gemm p, const Tile* tiles,
                                                             const int* ntiles) {
  static_assert(RG <= 8, "one scale block");
  // HBM is the bound, so sums are fp32 unless the result is rounded to e4m3
  // anyway (its eight row groups and both forms of the fragments need 263
  // registers: one work-group a CU, the decode batch's up projection 0.78 ms
  // against 0.575).
  constexpr bool EXACT = !std::is_same<OUT, Relu2Fp8>::value;
  __shared__ f32x4 red[NW][RG][64];
  const int nblocks = (p.N + 16 * RG - 1) / (16 * RG);
  const int nb = blockIdx.x % nblocks;
  const int tm = blockIdx.x / nblocks;
  int e = 0, m0 = 0, mcount = p.M;
  if (GROUPED) {
    if (tm >= *ntiles) return;
    e = uniform(tiles[tm].expert);
    m0 = uniform(tiles[tm].row0);
    mcount = uniform(tiles[tm].nrows);
  }
  const int n0 = nb * (16 * RG);
  const int lane = threadIdx.x & 63;
  const int w = uniform(threadIdx.x >> 6);
  const int r16 = lane & 15, kq = lane >> 4;
  const int K = p.K, KB = p.KB;
  const int kbeg = w * KB / NW, kend = (w + 1) * KB / NW;

  const int lrow = lane >> 3, lch = (lane & 7) * 16;
  const uint8_t* wa[RG];
  const uint8_t* wb[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g) {
    // 16-row groups past N read the last one (N is a multiple of 16)
    const int n = min(n0 + g * 16, p.N - 16);
    wa[g] = p.w + ((size_t)e * p.N + n + lrow) * K + lch;
    wb[g] = wa[g] + (size_t)8 * K;
  }
  // 16 RG rows lie in one scale block (RG <= 8 divides it)
  const float* wsp = p.ws + ((size_t)e * p.NB + n0 / 128) * KB;
  bool xok;
  const long row = fp8_x_row(p, m0 + (r16 < mcount ? r16 : 0), xok);
  const uint8_t* xp = p.x + row * K + kq * 16;
  const float* xsp = p.xs + row * KB;
  const int src0 = (((r16 & 7) << 3) | kq) * 4;
  const int src1 = (((r16 & 7) << 3) | (4 + kq)) * 4;
  const bool lo = r16 < 8;

  f32x4 acc[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g) acc[g] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Stage {
    i32x4 l[U][RG][2], x[U][2];
    float xs[U], ws[U];
  };
  auto load = [&](Stage& S, int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (U > 1 && kb + u >= kend) break;
      const int k = (kb + u) * 128;
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        S.l[u][g][0] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(wa[g] + k));
        S.l[u][g][1] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(wb[g] + k));
      }
      S.x[u][0] = *reinterpret_cast<const i32x4*>(xp + k);
      S.x[u][1] = *reinterpret_cast<const i32x4*>(xp + k + 64);
      S.xs[u] = xsp[kb + u];
      S.ws[u] = wsp[kb + u];
    }
  };
  auto compute = [&](const Stage& S, int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (U > 1 && kb + u >= kend) break;
      const Frag<EXACT> xf = as_frag<EXACT>(join(S.x[u][0], S.x[u][1]));
      const float f = (xok ? S.xs[u] : 0.f) * S.ws[u];
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        const i32x8 wf = join(fp8_permute(S.l[u][g][0], S.l[u][g][1], src0, lo),
                              fp8_permute(S.l[u][g][0], S.l[u][g][1], src1, lo));
        acc[g] += mfma_fp8(as_frag<EXACT>(wf), xf) * f;
      }
    }
  };
  Stage A, B;
  if (kbeg < kend) load(A, kbeg);
  for (int kb = kbeg; kb < kend; kb += 2 * U) {
    if (kb + U < kend) load(B, kb + U);
    compute(A, kb);
    if (kb + U < kend) {
      if (kb + 2 * U < kend) load(A, kb + 2 * U);
      compute(B, kb + U);
    }
  }

#pragma unroll
  for (int g = 0; g < RG; ++g) red[w][g][lane] = acc[g];
  __syncthreads();
  if constexpr (std::is_same<OUT, Relu2Fp8>::value) {
    // the work-group holds a whole block of 128 columns of each row
    static_assert(RG == 8 && RG % NW == 0, "one scale block");
    __shared__ float top[NW][16];
    f32x4 v[RG / NW];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < RG / NW; ++i) {
      const int g = w + i * NW;
      v[i] = red[0][g][lane];
#pragma unroll
      for (int u = 1; u < NW; ++u) v[i] += red[u][g][lane];
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, v[i][j] = relu_sq(v[i][j]));
    }
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    if (kq == 0) top[w][r16] = m;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NW; ++u) m = fmaxf(m, top[u][r16]);
    const float sc = fp8_scale(m);
    if (r16 < mcount) {
#pragma unroll
      for (int i = 0; i < RG / NW; ++i)
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.y) + (size_t)(m0 + r16) * p.N + n0 +
                                     (w + i * NW) * 16 + kq * 4) = fp8_codes4(v[i], sc);
      if (w == 0 && kq == 0) p.ys[(size_t)(m0 + r16) * p.NB + n0 / 128] = sc;
    }
    return;
  }
  for (int g = w; g < RG; g += NW) {
    f32x4 sm = red[0][g][lane];
#pragma unroll
    for (int v = 1; v < NW; ++v) sm += red[v][g][lane];
    const int n = n0 + g * 16;
    if (r16 < mcount && n < p.N) fp8_store4<OUT>(p, m0 + r16, n + kq * 4, sm);
  }
}

// Many tokens: MFMA tiles of BM token rows x BN weight rows fed through LDS by
// direct global -> LDS copies.  One step is a block of k (128 bytes of a row)
// in two halves of the block's weight rows; each wave owns 16 TM token rows
// and 16 TH weight rows of each half, and holds the fragments it multiplies
// in registers.  A fragment's registers are read anew from LDS, for the next
// half, right after their last use, so no LDS read is waited for at the top
// of a step.  During step kb, LDS holds what is read in it (weight half 1 of
// kb, half 0 of kb + 1, token rows of kb + 1), and copies run into the places
// of what step kb - 1 read: token rows of kb + 2 and, with a ring of WD
// blocks of weights, half 1 of block kb + WD - 1 and half 0 of kb + WD.  One
// barrier a step; the copy instructions are spread over the MFMAs.  Expert
// weights come from HBM and take WD = 3 (the copies of the last step may
// still be in flight at the barrier), dense ones mostly from L2.
//
// Scales: the tile's weight scales are read into LDS once.  Token scales come
// eight blocks of k at a time (32 bytes of a row of scales), an eighth of the
// rows with each token block: one block at a time, every 4-byte load was a
// cache line of its own, half as many line requests as the data itself.
//
// 8192 x 10240 x 8192: 528 to 558 us, 2.46 to 2.60 PFLOP/s (a library's product
// of the same codes without scales: 505); 180224 rows over 512 experts, 2048 x
// 5120: 2.10 to 2.14 ms, 1.77 to 1.80 PFLOP/s.  A step of a 256 x 256 tile takes 1.59 us and a tile 6.4 us
// beside its steps (192 x 256 grouped: 1.28 to 1.44 and 5.8): first copies and
// the store of the result, which the next tile's work-group waits for.
//
// Split over k (dense, few tiles): work-group (x, y) computes tile x over the
// y-th part of the blocks and writes fp32 partial sums to part y of `y`.
template <bool GROUPED, int BM, int BN, int WM, int WD, bool EXACT, class OUT>
__device__ __forceinline__ void fp8_pipe_body(Fp8Gemm p, const Tile* tiles, const int* ntiles) {
  constexpr int BH = BN / 2, WN = 8 / WM, NW = 8;
  constexpr int TM = BM / WM / 16, TH = BH / WN / 16;
  constexpr int RPI = kFp8CopyRows, ROWB = 128;
  constexpr int NIA = BM / RPI / NW, NIH = BH / RPI / NW;  // copies a wave and unit
  constexpr int ABUF = BM * ROWB, HBUF = BH * ROWB;
  constexpr int NSB = BN / 128;  // scale blocks of the tile's weight rows
  static_assert(NIA * RPI * NW == BM && NIH * RPI * NW == BH && BM % 64 == 0, "rows per unit");
  // One LDS array: with several, the compiler tells them apart and then waits
  // for all copies in flight before every LDS read.
  constexpr int W00 = 2 * ABUF, XS0 = W00 + 2 * WD * HBUF, WS0 = XS0 + 2 * BM * 32;
  constexpr int SO0 = WS0 + NSB * kFp8MaxBlocks * 4, LDS = SO0 + BM * 4;
  static_assert(LDS <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) char smem[LDS];
  float* const sxs = reinterpret_cast<float*>(smem + XS0);  // [2][BM][8] token scales
  float* const sws = reinterpret_cast<float*>(smem + WS0);  // [NSB][blocks] weight scales
  uint32_t* const sso = reinterpret_cast<uint32_t*>(smem + SO0);  // [BM] rows' scale offsets

  int tm, nb;
  const int nblocks = (p.N + BN - 1) / BN;
  if (!work_item_uniform<GROUPED>(nblocks, p.M, BM, tiles, ntiles, tm, nb)) return;
  int e = 0, m0, mcount;
  if (GROUPED) {
    e = uniform(tiles[tm].expert);
    m0 = uniform(tiles[tm].row0);
    mcount = uniform(tiles[tm].nrows);
  } else {
    m0 = tm * BM;
    mcount = min(BM, p.M - m0);
  }
  const int n0 = nb * BN;
  const int lane = threadIdx.x & 63;
  const int w = uniform(threadIdx.x >> 6);
  const int wm = w / WN, wn = w % WN;
  const int K = p.K, KBT = p.KB;  // blocks of a whole row
  int kb0 = 0, KB = KBT;          // this work-group's: kb0 .. kb0 + KB - 1
  if (!GROUPED && p.splits > 1) {
    kb0 = blockIdx.y * KBT / p.splits;
    KB = (blockIdx.y + 1) * KBT / p.splits - kb0;
    p.y = static_cast<float*>(p.y) + (size_t)blockIdx.y * p.M * p.N;
  }

  // Copy sources: instruction j of wave w fills rows RPI (w + NW j) .. + 7 of
  // its buffer, written already swizzled (16-byte chunk c of row r in place
  // c ^ (r / 2) % 8).  Token rows past the tile's count are past the buffer's
  // bound and read as 0 (nothing is fetched, and products of zeros take less
  // power: 1% faster than reading the first row again where 11% of the rows
  // are such).  Weight rows past N read the matrix's last rows again (their
  // columns are not stored).
  const int lr = lane >> 3;
  const int sw = ((4 * (w & 1)) + (lr >> 1)) & 7;
  const uint32_t chunk = (uint32_t)(((lane & 7) ^ sw) * 16);
  const bool gather = p.rows != nullptr;
  const uint8_t* xbase = (gather ? p.x : p.x + (size_t)m0 * K) + kb0 * ROWB;
  const float* xsbase = (gather ? p.xs : p.xs + (size_t)m0 * KBT) + kb0;
  auto x_row = [&](int i, bool& ok) -> uint32_t {
    const int m = i < mcount ? i : 0;
    ok = true;
    return gather ? (uint32_t)fp8_x_row(p, m0 + m, ok) : (uint32_t)m;
  };
  const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(xbase);
  const __amdgpu_buffer_rsrc_t rs =
      buffer_rsrc(xsbase, (((size_t)p.x_rows - (gather ? 0 : m0)) * KBT - kb0) * 4);
  const size_t w0 = ((size_t)e * p.N + n0) * K + kb0 * ROWB;
  const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(
      p.w + w0, (size_t)(GROUPED ? p.groups : 1) * p.N * K - w0);
  uint32_t ao[NIA], bo = fp8_weight_lane(lane, chunk, (uint32_t)K);
#pragma unroll
  for (int j = 0; j < NIA; ++j) {
    bool ok;
    const int i = RPI * (w + NW * j) + lr;
    ao[j] = i < mcount ? x_row(i, ok) * (uint32_t)K + chunk : 0x80000000u;
    asm volatile("" : "+v"(ao[j]));  // one register: not half of a 64-bit product
  }
  asm volatile("" : "+v"(bo));
  for (int i = threadIdx.x; i < BM; i += 512) {
    bool ok;
    sso[i] = x_row(i, ok) * (uint32_t)KBT * 4u;
  }

  // copy instruction j of token block kb, of weight half h of block kb
  auto copy_x = [&](int kb, int j) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        ra, (lds_void*)(smem + (kb & 1) * ABUF + (w + NW * j) * RPI * ROWB), 16, ao[j], kb * ROWB,
        0, 0);
  };
  // (to ring offset r)
  auto copy_w = [&](int kb, int h, int r, int j) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rb, (lds_void*)(smem + W00 + r + h * HBUF + (w + NW * j) * RPI * ROWB), 16, bo,
        fp8_weight_scalar(h * BH + (w + NW * j) * RPI, p.N - n0, kb, K), 0, 0);
  };
  // Token scales of blocks 8 g .. 8 g + 7: instruction i fills rows 8 i .. + 7,
  // lane l row 8 i + l / 8, place l % 8, which holds block (l % 8) ^ 4 (i % 2)
  // of the eight (so that 16 rows' reads of one block meet no bank twice).
  // Eighth j of a group is BM / 64 instructions, one a wave (some twice).
  // Blocks past K read the next row's scales, or 0 past the last one's;
  // nothing uses them.
  const int sg = w % (BM / 64);
  auto xs_row = [&](int j) __attribute__((always_inline)) {
    return sso[8 * (j * (BM / 64) + sg) + lr];
  };
  auto copy_xs = [&](int g, int j, uint32_t row) __attribute__((always_inline)) {
    const int i = j * (BM / 64) + sg;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rs, (lds_void*)(sxs + ((g & 1) * BM + 8 * i) * 8), 4,
        fp8_xscale_lane(row, lane, i, g), 0, 0, 0);
  };
  // weight scales of the tile: wave w takes 64 blocks of one of its 128-row
  // blocks (places past K hold what follows in memory, or 0 past its end)
  {
    static_assert(NSB * (kFp8MaxBlocks / 64) <= NW, "a wave for each 64 scales");
    const size_t ws0 = ((size_t)e * p.NB + n0 / 128) * KBT + kb0;
    const __amdgpu_buffer_rsrc_t rws =
        buffer_rsrc(p.ws + ws0, ((size_t)(GROUPED ? p.groups : 1) * p.NB * KBT - ws0) * 4);
    const int b = w % NSB, i = w / NSB;
    if (i < kFp8MaxBlocks / 64)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rws, (lds_void*)(sws + b * kFp8MaxBlocks + i * 64), 4,
          fp8_wscale_lane(lane, b, i, KBT), 0, 0, 0);
  }
  // what the first MFMAs need, then what step 0 reads, then what it need not
  // wait for
  constexpr int R = 2 * HBUF;  // a block's place in the ring of weights
#pragma unroll
  for (int j = 0; j < NIA; ++j) copy_x(0, j);
#pragma unroll
  for (int j = 0; j < NIH; ++j) copy_w(0, 0, 0, j);
  wait_lgkmcnt0();
  stage_barrier_hard();
#pragma unroll
  for (int j = 0; j < 8; ++j) copy_xs(0, j, xs_row(j));
#pragma unroll
  for (int j = 0; j < NIH; ++j) copy_w(0, 1, 0, j);
  if (KB > 1) {
#pragma unroll
    for (int j = 0; j < NIH; ++j) copy_w(1, 0, R, j);
#pragma unroll
    for (int j = 0; j < NIA; ++j) copy_x(1, j);
    copy_xs(1, 0, xs_row(0));
    if constexpr (WD == 3) {
#pragma unroll
      for (int j = 0; j < NIH; ++j) copy_w(1, 1, R, j);
      if (KB > 2) {
#pragma unroll
        for (int j = 0; j < NIH; ++j) copy_w(2, 0, 2 * R, j);
      }
    }
  }

  const int r16 = lane & 15, kq = lane >> 4;
  const uint32_t l0 = r16 * ROWB + (((0 + kq) ^ (r16 >> 1)) << 4);
  const uint32_t l1 = r16 * ROWB + (((4 + kq) ^ (r16 >> 1)) << 4);
  const uint32_t aw = (uint32_t)(wm * (BM / WM)) * ROWB;
  const uint32_t bw = (uint32_t)(W00 + wn * (BH / WN) * ROWB);
  // scale block of this wave's weight rows in each half
  const float* const wsl[2] = {sws + (wn * (BH / WN)) / 128 * kFp8MaxBlocks,
                               sws + (BH + wn * (BH / WN)) / 128 * kFp8MaxBlocks};
  f32x4 acc[2 * TH][TM];
#pragma unroll
  for (int a = 0; a < 2 * TH; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint32_t live = 0;  // token groups whose row index was in range
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    bool ok;
    (void)x_row(wm * (BM / WM) + t * 16 + r16, ok);
    live |= (uint32_t)ok << t;
  }

  // fragments: token group t of block kb, weight group g at ring offset r
  auto read_x = [&](int kb, int t) __attribute__((always_inline)) {
    const char* st = smem + (kb & 1) * ABUF + aw + t * 16 * ROWB;
    return join(*reinterpret_cast<const i32x4*>(st + l0), *reinterpret_cast<const i32x4*>(st + l1));
  };
  auto read_w = [&](int r, int g) __attribute__((always_inline)) {
    const char* st = smem + bw + r + g * 16 * ROWB;
    return join(*reinterpret_cast<const i32x4*>(st + l0), *reinterpret_cast<const i32x4*>(st + l1));
  };
  auto read_xs = [&](int kb, int t) __attribute__((always_inline)) {
    const int row = wm * (BM / WM) + t * 16 + r16;
    const float x = sxs[(((kb >> 3) & 1) * BM + row) * 8 + ((kb & 7) ^ ((row >> 1) & 4))];
    return (live >> t) & 1 ? x : 0.f;
  };
  i32x8 xf[TM], wf[TH];  // the current half's fragments
  float xs[TM];          // and the block's token scales

  int r0 = 0;  // ring offset of block kb
  // Step kb.  COPY: 2 copies everything (kb + WD < KB), 1 all but the weights
  // of block kb + WD (the last step with copies), 0 nothing.
  auto step = [&](auto copy_c, int kb) __attribute__((always_inline)) {
    constexpr int COPY = decltype(copy_c)::value;
    const int r1 = r0 + R == WD * R ? 0 : r0 + R;
    const int r2 = r1 + R == WD * R ? 0 : r1 + R;  // r0 when WD = 2
    // what this step reads has landed (with WD = 3 the weight copies of the
    // last step may be in flight), and this wave's LDS reads of the last step
    // are done; then the same for every wave
    if (WD == 3 && COPY) wait_vmcnt<2 * NIH>();
    else wait_vmcnt<0>();
    wait_lgkmcnt0();
    stage_barrier_hard();
    // the scales with token block n = kb + 2 are eighth (n - 1) % 8 of the
    // group that block n + 7 lies in, whose last eighth so comes with its
    // first block
    constexpr bool XC = COPY == 2 || (COPY == 1 && WD == 3);  // block kb + 2 exists
    constexpr int NX = XC ? NIA + 1 : 0;
    constexpr int NC = NX + (COPY == 2 ? 2 * NIH : (COPY == 1 ? NIH : 0));
    uint32_t xrow = 0;
    if constexpr (XC) xrow = xs_row((kb + 1) & 7);
    // in the order they are waited for; with WD = 2 that is the same barrier
    // for all, and weights first, the larger part, measured 3% faster
    constexpr int X0 = WD == 2 ? NC - NX : 0, W0 = WD == 2 ? 0 : NX;
    auto copy = [&](int c) __attribute__((always_inline)) {
      if (c >= X0 && c < X0 + NX - 1) copy_x(kb + 2, c - X0);
      else if (c >= X0 && c < X0 + NX) copy_xs((kb + 9) >> 3, (kb + 1) & 7, xrow);
      else if (c < W0 + NIH) copy_w(kb + WD - 1, 1, WD == 2 ? r1 : r2, c - W0);
      else copy_w(kb + WD, 0, r0, c - W0 - NIH);
    };
    float f[2][TM];
    const float s0 = wsl[0][kb], s1 = wsl[1][kb];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      f[0][t] = xs[t] * s0;
      f[1][t] = xs[t] * s1;
    }
    // the products run LAG MFMAs ahead of their scaling
    constexpr int NP = TM * TH, LAG = 3;
    // a copy after every other MFMA, or each where there are few
    constexpr int EVERY = NC <= NP ? 2 : 1;
    static_assert(NC <= 2 * NP, "copies");
    f32x4 q[LAG];
    Frag<EXACT> xq[TM], wq;
#pragma unroll
    for (int t = 0; t < TM; ++t) xq[t] = as_frag<EXACT>(xf[t]);
#pragma unroll
    for (int i = 0; i < 2 * NP + LAG; ++i) {
      if (i >= LAG) {
        const int j = i - LAG, h = j / NP, g = j % NP / TM, t = j % TM;
        acc[h * TH + g][t] += q[j % LAG] * f[h][t];
        // keeps the scaling here: it must not sink past the barrier, where
        // all of the step's products would be live at once
        asm volatile("" : "+v"(acc[h * TH + g][t]));
      }
      if (i < 2 * NP) {
        const int h = i / NP, g = i % NP / TM, t = i % TM;
        if (t == 0) wq = as_frag<EXACT>(wf[g]);
        q[i % LAG] = mfma_fp8(wq, xq[t]);
        if (t == TM - 1) wf[g] = read_w(h == 0 ? r0 + HBUF : r1, g);
        if (h == 1 && g == TH - 1) xf[t] = read_x(kb + 1, t);
        if (i % EVERY == 0 && i / EVERY < NC) copy(i / EVERY);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int t = 0; t < TM; ++t) xs[t] = read_xs(kb + 1, t);
    r0 = r1;
  };
  if (KB > 2) wait_vmcnt<(WD == 3 ? 4 : 2) * NIH + NIA + 1>();
  else wait_vmcnt<0>();
  stage_barrier_hard();
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    xf[t] = read_x(0, t);
    xs[t] = read_xs(0, t);
  }
#pragma unroll
  for (int g = 0; g < TH; ++g) wf[g] = read_w(0, g);
  int kb = 0;
  for (; kb + WD < KB; ++kb) step(std::integral_constant<int, 2>{}, kb);
  if (kb + WD - 1 < KB) step(std::integral_constant<int, 1>{}, kb++);
  for (; kb < KB; ++kb) step(std::integral_constant<int, 0>{}, kb);
  // the last step read ahead (values that are not used): let the reads end
  // before the buffers are written below
  wait_lgkmcnt0();
  stage_barrier_hard();

  const int mr = wm * (BM / WM);
  if constexpr (std::is_same<OUT, Relu2Fp8>::value) {
    // Each half is one block of 128 columns, held by WN waves: they exchange
    // their rows' largest values through the weight ring, then put the codes
    // into the token buffers as rows of 256 bytes (16-byte chunk c of row r
    // in place c ^ r % 16), which leave as whole cache lines.
    static_assert(BN == 256, "two scale blocks");
    float* const top = reinterpret_cast<float*>(smem + W00);  // [2][WN][BM]
#pragma unroll
    for (int g = 0; g < 2 * TH; ++g)
#pragma unroll
      for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[g][t][j] = relu_sq(acc[g][t][j]);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        float m = 0.f;
#pragma unroll
        for (int g = 0; g < TH; ++g)
#pragma unroll
          for (int j = 0; j < 4; ++j) m = fmaxf(m, acc[h * TH + g][t][j]);
        m = fmaxf(m, __shfl_xor(m, 16, 64));
        m = fmaxf(m, __shfl_xor(m, 32, 64));
        if (kq == 0) top[(h * WN + wn) * BM + mr + t * 16 + r16] = m;
      }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        const int row = mr + t * 16 + r16;
        float m = 0.f;
#pragma unroll
        for (int u = 0; u < WN; ++u) m = fmaxf(m, top[(h * WN + u) * BM + row]);
        const float sc = fp8_scale(m);
        if (wn == 0 && kq == 0 && row < mcount && n0 + h * 128 < p.N)
          p.ys[(size_t)(m0 + row) * p.NB + n0 / 128 + h] = sc;
#pragma unroll
        for (int g = 0; g < TH; ++g) {
          const int c = h * 8 + wn * TH + g;
          *reinterpret_cast<uint32_t*>(smem + row * 256 + ((c ^ r16) << 4) + kq * 4) =
              fp8_codes4(acc[h * TH + g][t], sc);
        }
      }
    __syncthreads();
    const int c = threadIdx.x & 15;
    for (int row = threadIdx.x >> 4; row < mcount; row += 32)
      if (n0 + c * 16 < p.N)
        *reinterpret_cast<i32x4*>(static_cast<uint8_t*>(p.y) + (size_t)(m0 + row) * p.N + n0 +
                                  c * 16) =
            *reinterpret_cast<const i32x4*>(smem + row * 256 + ((c ^ (row & 15)) << 4));
  } else if constexpr (std::is_same<OUT, uint16_t>::value) {
    // bf16 rows through LDS (staged_store), in the token buffers
    struct Out {
      const Fp8Gemm& p;
      __device__ u16x4 pack4(f32x4 v) const { return pack4_bf16(v); }
      __device__ void store8(int m, int n, u16x8 v) const {
        if (n < p.N)
          *reinterpret_cast<u16x8*>(static_cast<uint16_t*>(p.y) + (size_t)m * p.N + n) = v;
      }
    };
    constexpr int REG = 16 * TM * 32 * TH;
    static_assert(NW * REG <= 2 * ABUF, "staging room");
    char* const reg = smem + w * REG;
    const Out out{p};
    staged_store<TH, 0>(out, reg, lane, acc, m0 + mr, mcount - mr, n0 + wn * (BH / WN));
    staged_store<TH, TH>(out, reg, lane, acc, m0 + mr, mcount - mr, n0 + BH + wn * (BH / WN));
  } else {
#pragma unroll
    for (int g = 0; g < 2 * TH; ++g)
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        const int i = mr + t * 16 + r16;
        const int n = n0 + (g / TH) * BH + wn * (BH / WN) + (g % TH) * 16;
        if (i < mcount && n < p.N) fp8_store4<OUT>(p, m0 + i, n + kq * 4, acc[g][t]);
      }
  }
}

template <bool GROUPED, int BM, int BN, int WM, int WD, bool EXACT, class OUT>
__global__ __launch_bounds__(512) void fp8_pipe_kernel(Fp8Gemm p, const Tile* tiles,
                                                       const int* ntiles) {
  fp8_pipe_body<GROUPED, BM, BN, WM, WD, EXACT, OUT>(p, tiles, ntiles);
}

// y = the sum of the parts, in order, four values a thread.
__device__ __forceinline__ void put4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void put4(uint16_t* p, f32x4 v) { store4_bf16(p, v); }
template <class OUT>
__global__ __launch_bounds__(256) void fp8_add_kernel(const float* __restrict__ part, int splits,
                                                      long n4, OUT* __restrict__ y) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  f32x4 v = reinterpret_cast<const f32x4*>(part)[i];
  for (int s = 1; s < splits; ++s) v += reinterpret_cast<const f32x4*>(part)[s * n4 + i];
  put4(y + i * 4, v);
}

// ---- launchers ---------------------------------------------------------------------

namespace {

template <class F>
void with_input(bool bf16, bool vec, F f) {
  if (bf16 && vec) f(uint16_t{}, std::true_type{});
  else if (bf16) f(uint16_t{}, std::false_type{});
  else if (vec) f(float{}, std::true_type{});
  else f(float{}, std::false_type{});
}

bool wide(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// How a product runs.  Times below: 8192 tokens' and smaller problems of the
// layer's shapes (K = 8192, 2048 or 5120), one MI355X.
using Plan = Fp8Plan;

// Grouped: rows per group on average decide.  Up to 4, weights are streamed
// past 16-row tiles (decode, 1.4 rows: 589 us; at 8.3 rows 1009 us against
// 915 for 64-row tiles).  Above that, the tile height with the least work:
// a group of r rows takes about r / BM + 0.4 tiles (at least one), whose cost
// for 64, 128 and 192 rows is 1.0, 1.25 and 1.675 us a block of k on the full
// chip (44 rows a group: 1086 / 1123 / 1261 us; 88: 1472 / 1197 / 1289; 176:
// 2088 / 1856 / 1468; 352: - / 2403 / 2145).
Plan tiled_plan(double r) {
  const int bm[3] = {64, 128, 192};
  const double cost[3] = {1.0, 1.25, 1.675};
  int best = 0;
  double least = 0;
  for (int i = 0; i < 3; ++i) {
    const double n = r / bm[i] + 0.4;
    const double c = (n > 1 ? n : 1.0) * cost[i];
    if (i == 0 || c < least) best = i, least = c;
  }
  return {false, bm[best], 1};
}
Plan grouped_plan(int rows, int groups, int KB) {
  if (rows <= 4L * groups || KB > kFp8MaxBlocks) return {true, kStreamTileM, 1};
  return tiled_plan((double)rows / groups);
}

// Dense: up to 16 rows stream the weights (1 / 16 rows x 2048 x 8192: 9.5 / 10.3
// us a call, 17 in tiles 13.6; 1 / 4 / 8 / 16 rows x 10240 x 8192: 16.5 / 17.2 /
// 19.6 / 24.7, 17 in tiles 19.0: with that many work-groups, each reading all
// of x, tiles would win from about 8 rows on).  Above that the tile shape and the split of k with
// the least estimated time: rounds of tiles over the 256 CUs, each so many
// blocks of k long (256 x 256 tiles: 1.65 us a block, 128 x 256: 0.96; 64 x
// 128 tiles, two of which fit a CU: 0.36, or 0.34 for each 256 of them), plus
// what a tile takes to start and end and, for a split, the second launch and
// the partial sums' traffic.  187 x 2048 x 8192: 24 us unsplit, 14.6 in 4 parts,
// 16.7 in 8; 32 x 10240 x 8192: 31 unsplit, 19.5 in 4.  fp32 results (`exact`: twice the MFMA time and
// the conversions) run on the same estimate without 256 x 256 tiles, whose
// converted fragments do not fit the registers; the better of the other two
// is at most 12% faster than what that picks, from 17 rows to 8192 (8192 x
// 10240 x 8192: 1160 us, 1.19 PFLOP/s, against 543 in bf16).
struct DenseTile {
  int bm, bn;
};
constexpr DenseTile kDenseTiles[3] = {{256, 256}, {128, 256}, {64, 128}};
double tile_us(const DenseTile& t, long n) {
  if (t.bm == 64) return n * (0.34 / 256) > 0.36 ? n * (0.34 / 256) : 0.36;
  return (double)((n + 255) / 256) * (t.bm == 256 ? 1.65 : 0.96);
}
Plan dense_plan(int M, int N, int KB, bool exact) {
  if (M <= 16) return {true, kStreamTileM, 1};
  Plan best{};
  double least = 0;
  for (const DenseTile& t : kDenseTiles) {
    if (exact && t.bm == 256) continue;
    for (int s = 1; s <= 8; s *= 2) {
      // a part is at least 8 blocks, and at most what the kernel takes
      const int kb = (KB + s - 1) / s;
      if ((s > 1 && KB / s < 8) || kb > kFp8MaxBlocks) continue;
      const long n = (long)((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn) * s;
      double us = tile_us(t, n) * kb + 3.4;
      if (s > 1) us += 4.0 + (double)s * M * N * 8 / 4e6;
      if (best.bm == 0 || us < least) best = {false, t.bm, s}, least = us;
    }
  }
  return best;
}

Plan make_plan(int M, int N, int KB, int groups, bool exact) {
  return groups ? grouped_plan(M, groups, KB) : dense_plan(M, N, KB, exact);
}

int grouped_tiles(int rows, int groups, int tile_m) {
  return (rows < groups ? rows : groups) + rows / tile_m + 1;
}

long xcd_grid(long work) { return kXcds * ((work + kXcds - 1) / kXcds); }

// A launch has fewer than 2^32 threads.
bool too_many(long grid, int threads) { return grid >= (1L << 32) / threads; }

// Grouped launches: row groups of 16 weight rows that a streaming work-group
// takes (a whole block of 128 where it quantises its output), weight rows of a
// tile, threads and work-groups.
constexpr int stream_groups(bool quantised) { return quantised ? 8 : 4; }
constexpr int kStreamWaves = 4, kGroupedBN = 256, kTileThreads = 512;
long grouped_grid(const Plan& plan, long max_tiles, int N, bool quantised) {
  const int bn = plan.stream ? 16 * stream_groups(quantised) : kGroupedBN;
  const long work = max_tiles * ((N + bn - 1) / bn);
  return plan.stream ? work : xcd_grid(work);
}
bool grouped_fits(const Plan& plan, long max_tiles, int N, bool quantised) {
  return !too_many(grouped_grid(plan, max_tiles, N, quantised),
                   plan.stream ? kStreamWaves * 64 : kTileThreads);
}

// Four waves x 4 row groups: 589 and 559 us for the decode batch's up and down
// projection, against 644 and 557 for 8 x 2, 615 and 563 for 4 x 2, 928 and
// 601 for 8 x 1; 595 and 565 for 4 x 8, which quantises its output (all with the
// 8-bit sums; fp32 sums change 4 x 4 by less than these runs differ).
template <class OUT>
hipError_t launch_grouped(const Fp8Gemm& p, const Plan& plan, const Tile* tiles, const int* ntiles,
                          int max_tiles, hipStream_t s) {
  using std::integral_constant;
  constexpr bool Q = std::is_same<OUT, Relu2Fp8>::value;
  if (!grouped_fits(plan, max_tiles, p.N, Q)) return hipErrorInvalidConfiguration;
  const long grid = grouped_grid(plan, max_tiles, p.N, Q);
  if (plan.stream) {
    constexpr int RG = stream_groups(Q), NW = kStreamWaves;
    fp8_stream_kernel<true, NW, RG, 1, OUT><<<grid, NW * 64, 0, s>>>(p, tiles, ntiles);
  } else {
    auto go = [&](auto bm, auto wm) {
      fp8_pipe_kernel<true, decltype(bm)::value, kGroupedBN, decltype(wm)::value, 3,
                      std::is_same<OUT, float>::value, OUT>
          <<<grid, kTileThreads, 0, s>>>(p, tiles, ntiles);
    };
    if (plan.bm == 64) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (plan.bm == 128) go(integral_constant<int, 128>{}, integral_constant<int, 2>{});
    else go(integral_constant<int, 192>{}, integral_constant<int, 4>{});
  }
  return hipGetLastError();
}

template <bool EXACT, class OUT>
hipError_t launch_dense(const Fp8Gemm& p, const Plan& plan, hipStream_t s) {
  using std::integral_constant;
  if (plan.stream) {
    constexpr int RG = 1, NW = 8;
    const long grid = (p.N + 16 * RG - 1) / (16 * RG);
    fp8_stream_kernel<false, NW, RG, 2, OUT><<<grid, NW * 64, 0, s>>>(p, nullptr, nullptr);
  } else {
    auto go = [&](auto bm, auto bn, auto wm, auto wd) {
      constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value;
      const long tot = (long)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
      fp8_pipe_kernel<false, BM, BN, decltype(wm)::value, decltype(wd)::value, EXACT, OUT>
          <<<dim3(xcd_grid(tot), p.splits), 512, 0, s>>>(p, nullptr, nullptr);
    };
    using I2 = integral_constant<int, 2>;
    using I3 = integral_constant<int, 3>;
    using I4 = integral_constant<int, 4>;
    using I128 = integral_constant<int, 128>;
    using I256 = integral_constant<int, 256>;
    if constexpr (!EXACT)
      if (plan.bm == 256) go(I256{}, I256{}, I4{}, I2{});
    if (plan.bm == 128) go(I128{}, I256{}, I2{}, I3{});
    else if (plan.bm == 64) go(integral_constant<int, 64>{}, I128{}, I2{}, I3{});
  }
  return hipGetLastError();
}

}  // namespace

hipError_t fp8_quantize(const void* x, bool bf16, long rows, int cols, long stride,
                        uint8_t* codes, float* scales, hipStream_t s) {
  const int nb = (cols + 127) / 128;
  const long grid = (rows * nb + 15) / 16;
  const bool vec = cols % 8 == 0 && stride % (bf16 ? 8 : 4) == 0 && wide(x, 16) && wide(codes, 8);
  with_input(bf16, vec, [&](auto t, auto v) {
    using T = decltype(t);
    fp8_quantize_kernel<T, decltype(v)::value><<<grid, 256, 0, s>>>(
        static_cast<const T*>(x), rows, cols, stride, nb, codes, scales);
  });
  return hipGetLastError();
}

hipError_t fp8_quantize_weight(const void* w, bool bf16, long matrices, int rows, int cols,
                               uint8_t* codes, float* scales, hipStream_t s) {
  const int rb = (rows + 127) / 128, cb = (cols + 127) / 128;
  const long grid = matrices * rb * cb;
  const bool vec = cols % 8 == 0 && wide(w, 16) && wide(codes, 8);
  with_input(bf16, vec, [&](auto t, auto v) {
    using T = decltype(t);
    fp8_quantize_weight_kernel<T, decltype(v)::value><<<grid, 256, 0, s>>>(
        static_cast<const T*>(w), rows, cols, rb, cb, codes, scales);
  });
  return hipGetLastError();
}

bool fp8_matmul_fits(int M, int N, int KB, int groups, bool out_bf16) {
  const Plan plan = make_plan(M, N, KB, groups, !out_bf16);
  if (groups) return grouped_fits(plan, grouped_tiles(M, groups, plan.bm), N, false);
  if (plan.stream) return true;  // up to 16 rows
  const int bn = plan.bm == 64 ? 128 : 256;
  return !too_many(xcd_grid((long)((M + plan.bm - 1) / plan.bm) * ((N + bn - 1) / bn)),
                   kTileThreads);
}

size_t fp8_matmul_workspace(int M, int N, int KB, int groups, bool out_bf16) {
  const Plan plan = make_plan(M, N, KB, groups, !out_bf16);
  if (groups) return 256 + (size_t)grouped_tiles(M, groups, plan.bm) * sizeof(Tile);
  return plan.splits > 1 ? (size_t)plan.splits * M * N * sizeof(float) : 0;
}

hipError_t fp8_matmul(Fp8Gemm p, const int32_t* offsets, bool out_bf16, void* ws, hipStream_t s) {
  const Plan plan = make_plan(p.M, p.N, p.KB, p.groups, !out_bf16);
  p.splits = plan.splits;
  if (p.groups) {
    const int max_tiles = grouped_tiles(p.M, p.groups, plan.bm);
    int32_t* ntiles = static_cast<int32_t*>(ws);
    Tile* tiles = reinterpret_cast<Tile*>(static_cast<char*>(ws) + 256);
    fp8_tiles_kernel<<<1, 1024, 0, s>>>(offsets, p.groups, p.M, plan.bm, max_tiles, tiles, ntiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return out_bf16 ? launch_grouped<uint16_t>(p, plan, tiles, ntiles, max_tiles, s)
                    : launch_grouped<float>(p, plan, tiles, ntiles, max_tiles, s);
  }
  if (p.splits > 1) {
    void* y = p.y;
    p.y = ws;
    const hipError_t e =
        out_bf16 ? launch_dense<false, float>(p, plan, s) : launch_dense<true, float>(p, plan, s);
    if (e != hipSuccess) return e;
    const long n4 = (long)p.M * p.N / 4;
    const long grid = (n4 + 255) / 256;
    const float* part = static_cast<const float*>(ws);
    if (out_bf16)
      fp8_add_kernel<<<grid, 256, 0, s>>>(part, p.splits, n4, static_cast<uint16_t*>(y));
    else
      fp8_add_kernel<<<grid, 256, 0, s>>>(part, p.splits, n4, static_cast<float*>(y));
    return hipGetLastError();
  }
  return out_bf16 ? launch_dense<false, uint16_t>(p, plan, s)
                  : launch_dense<true, float>(p, plan, s);
}

Fp8Plan fp8_expert_plan(int rows, int experts, int KB, int path) {
  if (KB > kFp8MaxBlocks || path == 1) return {true, kStreamTileM, 1};
  return path == 2 ? tiled_plan((double)rows / experts) : grouped_plan(rows, experts, KB);
}

bool fp8_experts_fit(const Fp8Plan& plan, long max_tiles, int F, int R) {
  return grouped_fits(plan, max_tiles, F, true) && grouped_fits(plan, max_tiles, R, false);
}

hipError_t fp8_exp_up(const Fp8Gemm& p, const Fp8Plan& plan, const Tile* tiles, const int* ntiles,
                      int max_tiles, hipStream_t s) {
  return launch_grouped<Relu2Fp8>(p, plan, tiles, ntiles, max_tiles, s);
}

hipError_t fp8_exp_down(const Fp8Gemm& p, const Fp8Plan& plan, const Tile* tiles,
                        const int* ntiles, int max_tiles, hipStream_t s) {
  return launch_grouped<uint16_t>(p, plan, tiles, ntiles, max_tiles, s);
}

}  // namespace lmoe
