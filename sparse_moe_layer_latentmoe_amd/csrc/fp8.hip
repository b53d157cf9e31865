// Matrices in 8-bit floating point (e4m3, OCP: largest finite value 448) with
// an fp32 scale for each block of 128 along k, and their products.
//
//   activations x [M, K]: scale xs[m][k / 128]; weights w [N, K]: scale
//   ws[n / 128][k / 128].  value = code * scale.
//   y[m][n] = sum over blocks b of xs[m][b] ws[n / 128][b] (sum of codes' products)
//
// Each block's sum of code products is one MFMA 16x16x128 from a zero
// accumulator; it is scaled in fp32 into the running sum (four fused
// multiply-adds per MFMA and lane, which run beside the next MFMA).  Weights
// are the MFMA's A operand and tokens its B operand, so a lane's four results
// are consecutive columns of one token and the scale is one factor per lane.
//
// A fragment is 32 bytes of a row; which k a lane holds does not matter as
// long as both operands agree, so lane (r, q) (r = lane % 16, q = lane / 16)
// takes the 16-byte chunks q and 4 + q of row r's 128 bytes.
#include <type_traits>

#include "fp8_device.h"
#include "gemm_device.h"
#include "kernels.h"

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
// very small scales take the division itself.
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
    for (int i = 0; i < 8; ++i) q[i] = fp8_ratio(v[i], s, r);
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
  float m = max8(v);
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  const float s = fp8_scale(m);
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
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
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
    n = max(min(offsets[g + 1], rows) - beg, 0);
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

template <class OUT>
__device__ __forceinline__ void fp8_store4(const Fp8Gemm& p, int m, int n, f32x4 v) {
  OUT* y = static_cast<OUT*>(p.y) + (size_t)m * p.N + n;
  if constexpr (std::is_same<OUT, float>::value)
    *reinterpret_cast<f32x4*>(y) = v;
  else
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
// GEMM measured fastest).  Work-group: 16 RG weight rows x 16 MT token rows.
template <bool GROUPED, int NW, int MT, int RG, int U, class OUT>
__global__ __launch_bounds__(NW * 64) void fp8_stream_kernel(Fp8Gemm p, const Tile* tiles,
                                                             const int* ntiles) {
  constexpr int J = RG * MT;
  __shared__ f32x4 red[NW > 1 ? NW : 1][J][64];
  const int nblocks = (p.N + 16 * RG - 1) / (16 * RG);
  int nb, tm;
  if (GROUPED) {
    nb = blockIdx.x % nblocks;
    tm = blockIdx.x / nblocks;
  } else {
    // the m tiles that share a weight block run back to back on one XCD
    const int mtiles = (p.M + 16 * MT - 1) / (16 * MT);
    const int local = blockIdx.x / kXcds;
    tm = local % mtiles;
    nb = (local / mtiles) * kXcds + blockIdx.x % kXcds;
    if (nb >= nblocks) return;
  }
  int e = 0, m0, mcount;
  if (GROUPED) {
    if (tm >= *ntiles) return;
    e = uniform(tiles[tm].expert);
    m0 = uniform(tiles[tm].row0);
    mcount = uniform(tiles[tm].nrows);
  } else {
    m0 = tm * (16 * MT);
    mcount = min(16 * MT, p.M - m0);
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
  const uint8_t* xp[MT];
  const float* xsp[MT];
  bool xok[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int i = t * 16 + r16;
    const long row = fp8_x_row(p, m0 + (i < mcount ? i : 0), xok[t]);
    xp[t] = p.x + row * K + kq * 16;
    xsp[t] = p.xs + row * KB;
  }
  const int src0 = (((r16 & 7) << 3) | kq) * 4;
  const int src1 = (((r16 & 7) << 3) | (4 + kq)) * 4;
  const bool lo = r16 < 8;

  f32x4 acc[RG][MT];
#pragma unroll
  for (int g = 0; g < RG; ++g)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[g][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Stage {
    i32x4 l[U][RG][2], x[U][MT][2];
    float xs[U][MT], ws[U];
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
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        S.x[u][t][0] = *reinterpret_cast<const i32x4*>(xp[t] + k);
        S.x[u][t][1] = *reinterpret_cast<const i32x4*>(xp[t] + k + 64);
        S.xs[u][t] = xsp[t][kb + u];
      }
      S.ws[u] = wsp[kb + u];
    }
  };
  auto compute = [&](const Stage& S, int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (U > 1 && kb + u >= kend) break;
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        const i32x8 wf = join(fp8_permute(S.l[u][g][0], S.l[u][g][1], src0, lo),
                              fp8_permute(S.l[u][g][0], S.l[u][g][1], src1, lo));
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const f32x4 q = mfma_fp8(wf, join(S.x[u][t][0], S.x[u][t][1]));
          const float f = (xok[t] ? S.xs[u][t] : 0.f) * S.ws[u];
          acc[g][t] += q * f;
        }
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

  if constexpr (NW > 1) {
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
      for (int t = 0; t < MT; ++t) red[w][g * MT + t][lane] = acc[g][t];
    __syncthreads();
    for (int j = w; j < J; j += NW) {
      f32x4 sm = red[0][j][lane];
#pragma unroll
      for (int v = 1; v < NW; ++v) sm += red[v][j][lane];
      const int g = j / MT, t = j % MT;
      const int i = t * 16 + r16, n = n0 + g * 16;
      if (i < mcount && n < p.N) fp8_store4<OUT>(p, m0 + i, n + kq * 4, sm);
    }
  } else {
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int i = t * 16 + r16, n = n0 + g * 16;
        if (i < mcount && n < p.N) fp8_store4<OUT>(p, m0 + i, n + kq * 4, acc[g][t]);
      }
  }
}

// Many tokens: the half-step pipeline of the bf16 GEMM (lds_pipe_kernel in
// gemm_tiled.hip) on rows of 128 bytes = one block of k.  Half-step s = 2 kb
// + h multiplies block kb of the token rows with half h of the block's weight
// rows; copy units (a weight half, plus the token rows and their scales when
// h = 0) are issued three half-steps ahead, so the copy stream never drains.
// Four half-steps are written out, so that every LDS address is a constant,
// and all but the last few run without conditions.
// Eight waves, WM along tokens x 8 / WM along weights.  The weight scales of
// the whole tile are read into LDS once.
template <bool GROUPED, int BM, int BN, int WM, class OUT>
__device__ __forceinline__ void fp8_pipe_body(const Fp8Gemm& p, const Tile* tiles,
                                              const int* ntiles) {
  constexpr int BH = BN / 2, WN = 8 / WM, NW = 8;
  constexpr int TM = BM / WM / 16, TH = BH / WN / 16;
  constexpr int RPI = 8, ROWB = 128;
  constexpr int NIA = BM / RPI / NW, NIH = BH / RPI / NW, NI0 = NIA + 1 + NIH;
  constexpr int L = 3, NBUF = L + 1;  // copy units in flight, weight-half buffers
  constexpr int ABUF = BM * ROWB, HBUF = BH * ROWB;
  constexpr int NSB = BN / 128;  // scale blocks of the tile's weight rows
  static_assert(NIA * RPI * NW == BM && NIH * RPI * NW == BH && BM % 64 == 0, "rows per unit");
  // One LDS array: with several, the compiler tells them apart and then waits
  // for all copies in flight before every LDS read.
  constexpr int XS0 = 2 * ABUF + NBUF * HBUF, WS0 = XS0 + 2 * BM * 4;
  __shared__ __attribute__((aligned(1024))) char smem[WS0 + NSB * kFp8MaxBlocks * 4];
  float* const sxs = reinterpret_cast<float*>(smem + XS0);  // [2][BM] token scales
  float* const sws = reinterpret_cast<float*>(smem + WS0);  // [NSB][blocks] weight scales

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
  const int K = p.K, KB = p.KB;
  const int nsub = 2 * KB;

  // Copy sources: instruction j of wave w fills rows RPI (w + NW j) .. + 7 of
  // its buffer, written already swizzled (16-byte chunk c of row r in place
  // c ^ (r / 2) % 8); token rows past the tile's count read its first row,
  // weight rows past N the last one.
  const int lr = lane >> 3;
  const int sw = ((4 * (w & 1)) + (lr >> 1)) & 7;
  const uint32_t chunk = (uint32_t)(((lane & 7) ^ sw) * 16);
  const bool gather = p.rows != nullptr;
  const uint8_t* xbase = gather ? p.x : p.x + (size_t)m0 * K;
  const float* xsbase = gather ? p.xs : p.xs + (size_t)m0 * KB;
  auto x_row = [&](int i, bool& ok) -> uint32_t {
    const int m = i < mcount ? i : 0;
    ok = true;
    return gather ? (uint32_t)fp8_x_row(p, m0 + m, ok) : (uint32_t)m;
  };
  const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(xbase), rs = buffer_rsrc(xsbase);
  const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(p.w + ((size_t)e * p.N + n0) * K);
  uint32_t ao[NIA], bo[2][NIH];
#pragma unroll
  for (int j = 0; j < NIA; ++j) {
    bool ok;
    ao[j] = x_row(RPI * (w + NW * j) + lr, ok) * (uint32_t)K + chunk;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < NIH; ++j)
      bo[h][j] = (uint32_t)(min(n0 + h * BH + RPI * (w + NW * j) + lr, p.N - 1) - n0) *
                     (uint32_t)K + chunk;
  // token scales: 64 a wave and instruction (waves beyond BM / 64 repeat)
  const int sg = w % (BM / 64);
  bool dummy;
  const uint32_t so = x_row(sg * 64 + lane, dummy) * (uint32_t)KB * 4u;

  // copy unit u (half H of block u / 2, into weight buffer WB)
  auto issue = [&](auto h_c, auto wb_c, int u) __attribute__((always_inline)) {
    constexpr int H = decltype(h_c)::value, WB = decltype(wb_c)::value & 3, AB = WB >> 1;
    const int kb = u >> 1;
    if constexpr (H == 0) {
      char* st = smem + AB * ABUF;
#pragma unroll
      for (int j = 0; j < NIA; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(st + (w + NW * j) * RPI * ROWB),
                                                 16, ao[j], kb * ROWB, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(sxs + AB * BM + sg * 64), 4, so, kb * 4,
                                               0, 0);
    }
    char* st = smem + 2 * ABUF + WB * HBUF;
#pragma unroll
    for (int j = 0; j < NIH; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(st + (w + NW * j) * RPI * ROWB), 16,
                                               bo[H][j], kb * ROWB, 0, 0);
  };
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
  using C3 = std::integral_constant<int, 3>;
  issue(C0{}, C0{}, 0);
  issue(C1{}, C1{}, 1);
  if (nsub > 2) issue(C0{}, C2{}, 2);
  // the tile's weight scales, written to LDS before the first barrier
  for (int i = threadIdx.x; i < NSB * KB; i += 512) {
    const int b = i / KB, k = i - b * KB;
    sws[b * kFp8MaxBlocks + k] =
        p.ws[((size_t)e * p.NB + min(n0 / 128 + b, p.NB - 1)) * KB + k];
  }
  wait_lgkmcnt0();

  const int r16 = lane & 15, kq = lane >> 4;
  const uint32_t l0 = r16 * ROWB + (((0 + kq) ^ (r16 >> 1)) << 4);
  const uint32_t l1 = r16 * ROWB + (((4 + kq) ^ (r16 >> 1)) << 4);
  const uint32_t aw = (uint32_t)(wm * (BM / WM)) * ROWB;
  const uint32_t bw = (uint32_t)(wn * (BH / WN)) * ROWB;
  // scale block of this wave's weight rows in each half
  const float* const wsl[2] = {sws + (wn * (BH / WN)) / 128 * kFp8MaxBlocks,
                               sws + (BH + wn * (BH / WN)) / 128 * kFp8MaxBlocks};
  f32x4 acc[2 * TH][TM];
#pragma unroll
  for (int a = 0; a < 2 * TH; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  i32x8 xf[TM];  // token fragments of the current block of k, and their scales
  float xs[TM];
  uint32_t live = 0;  // token groups whose row index was in range
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    bool ok;
    (void)x_row(wm * (BM / WM) + t * 16 + r16, ok);
    live |= (uint32_t)ok << t;
  }

  // half-step s with s % 4 = S4; MORE: units s + 1 .. s + L all exist
  auto half_step = [&](auto s4_c, auto more_c, int s) __attribute__((always_inline)) {
    constexpr int S4 = decltype(s4_c)::value, H = S4 & 1, AB = S4 >> 1;
    constexpr bool MORE = decltype(more_c)::value;
    // unit s has landed: at most units s + 1 and s + 2 are still in flight
    if (MORE || s + 2 < nsub) wait_vmcnt<NI0 + NIH>();
    else if (H == 0 && s + 1 < nsub) wait_vmcnt<NIH>();
    else wait_vmcnt<0>();
    stage_barrier_hard();
    if (MORE || s + L < nsub)
      issue(std::integral_constant<int, H ^ 1>{}, std::integral_constant<int, (S4 + L) & 3>{},
            s + L);
    const int kb = s >> 1;
    if constexpr (H == 0) {
      const char* st = smem + AB * ABUF + aw;
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        xf[t] = join(*reinterpret_cast<const i32x4*>(st + l0 + t * 16 * ROWB),
                     *reinterpret_cast<const i32x4*>(st + l1 + t * 16 * ROWB));
        const float v = sxs[AB * BM + wm * (BM / WM) + t * 16 + r16];
        xs[t] = (live >> t) & 1 ? v : 0.f;
      }
    }
    const char* st = smem + 2 * ABUF + S4 * HBUF + bw;
    i32x8 wf[TH];
#pragma unroll
    for (int g = 0; g < TH; ++g)
      wf[g] = join(*reinterpret_cast<const i32x4*>(st + l0 + g * 16 * ROWB),
                   *reinterpret_cast<const i32x4*>(st + l1 + g * 16 * ROWB));
    const float ws = wsl[H][kb];
    // the products run AHEAD MFMAs ahead of their scaling
    constexpr int NP = TM * TH, AHEAD = 3;
    f32x4 q[AHEAD];
    float f = 0.f;
#pragma unroll
    for (int i = 0; i < NP + AHEAD; ++i) {
      if (i >= AHEAD) {
        const int t = (i - AHEAD) / TH, g = (i - AHEAD) % TH;
        if (g == 0) f = xs[t] * ws;
        acc[H * TH + g][t] += q[i % AHEAD] * f;
        // keeps the scaling here: it must not sink past the barrier, where
        // all of the half-step's products would be live at once
        asm volatile("" : "+v"(acc[H * TH + g][t]));
      }
      if (i < NP) q[i % AHEAD] = mfma_fp8(wf[i % TH], xf[i / TH]);
    }
  };
  int s = 0;
  for (; s + 3 + L < nsub; s += 4) {
    half_step(C0{}, std::true_type{}, s);
    half_step(C1{}, std::true_type{}, s + 1);
    half_step(C2{}, std::true_type{}, s + 2);
    half_step(C3{}, std::true_type{}, s + 3);
  }
  for (; s < nsub; s += 4) {
    half_step(C0{}, std::false_type{}, s);
    half_step(C1{}, std::false_type{}, s + 1);
    if (s + 2 < nsub) {
      half_step(C2{}, std::false_type{}, s + 2);
      half_step(C3{}, std::false_type{}, s + 3);
    }
  }

  const int wr = wm * (BM / WM);
  if constexpr (std::is_same<OUT, uint16_t>::value) {
    // bf16 rows through LDS (staged_store), in the token buffers: their last
    // readers passed the last half-step's barrier, and every copy has landed
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
    staged_store<TH, 0>(out, reg, lane, acc, m0 + wr, mcount - wr, n0 + wn * (BH / WN));
    staged_store<TH, TH>(out, reg, lane, acc, m0 + wr, mcount - wr, n0 + BH + wn * (BH / WN));
  } else {
#pragma unroll
    for (int g = 0; g < 2 * TH; ++g)
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        const int i = wr + t * 16 + r16;
        const int n = n0 + (g / TH) * BH + wn * (BH / WN) + (g % TH) * 16;
        if (i < mcount && n < p.N) fp8_store4<OUT>(p, m0 + i, n + kq * 4, acc[g][t]);
      }
  }
}

template <bool GROUPED, int BM, int BN, int WM, class OUT>
__global__ __launch_bounds__(512) void fp8_pipe_kernel(Fp8Gemm p, const Tile* tiles,
                                                       const int* ntiles) {
  fp8_pipe_body<GROUPED, BM, BN, WM, OUT>(p, tiles, ntiles);
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

// Rows per group (average) up to which a grouped product streams weights,
// and rows up to which a dense one does.
constexpr int kStreamGroupRows = 32;
constexpr int kStreamRows = 64;

template <class OUT>
hipError_t launch(const Fp8Gemm& p, const Tile* tiles, const int* ntiles, int max_tiles,
                  bool stream, hipStream_t s) {
  if (p.groups) {
    if (stream) {
      constexpr int RG = 2, NW = 8;
      const long grid = (long)max_tiles * ((p.N + 16 * RG - 1) / (16 * RG));
      fp8_stream_kernel<true, NW, 1, RG, 1, OUT><<<grid, NW * 64, 0, s>>>(p, tiles, ntiles);
    } else {
      constexpr int BN = 256;
      const long grid = kXcds * (((long)max_tiles * ((p.N + BN - 1) / BN) + kXcds - 1) / kXcds);
      fp8_pipe_kernel<true, kFp8TileM, BN, 2, OUT><<<grid, 512, 0, s>>>(p, tiles, ntiles);
    }
    return hipGetLastError();
  }
  if (stream) {
    auto go = [&](auto mt) {
      constexpr int MT = decltype(mt)::value, RG = 1, NW = 8;
      const long nblocks = (p.N + 16 * RG - 1) / (16 * RG);
      const long mtiles = (p.M + 16 * MT - 1) / (16 * MT);
      const long grid = kXcds * mtiles * ((nblocks + kXcds - 1) / kXcds);
      fp8_stream_kernel<false, NW, MT, RG, 2, OUT><<<grid, NW * 64, 0, s>>>(p, nullptr, nullptr);
    };
    if (p.M <= 16) go(std::integral_constant<int, 1>{});
    else if (p.M <= 32) go(std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 4>{});
    return hipGetLastError();
  }
  constexpr int BM = 256, BN = 256;
  const long tot = (long)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  const long grid = kXcds * ((tot + kXcds - 1) / kXcds);
  fp8_pipe_kernel<false, BM, BN, 4, OUT><<<grid, 512, 0, s>>>(p, nullptr, nullptr);
  return hipGetLastError();
}

bool grouped_stream(int rows, int groups) { return rows <= (long)kStreamGroupRows * groups; }

int grouped_tiles(int rows, int groups, int tile_m) {
  return (rows < groups ? rows : groups) + rows / tile_m + 1;
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

size_t fp8_matmul_workspace(int rows, int groups) {
  if (groups == 0) return 0;
  const int tile_m = grouped_stream(rows, groups) ? kStreamTileM : kFp8TileM;
  return 256 + (size_t)grouped_tiles(rows, groups, tile_m) * sizeof(Tile);
}

hipError_t fp8_matmul(const Fp8Gemm& p, const int32_t* offsets, bool out_bf16, void* ws,
                      hipStream_t s) {
  Tile* tiles = nullptr;
  int32_t* ntiles = nullptr;
  int max_tiles = 0;
  bool stream = p.M <= kStreamRows;
  if (p.groups) {
    stream = grouped_stream(p.M, p.groups);
    const int tile_m = stream ? kStreamTileM : kFp8TileM;
    max_tiles = grouped_tiles(p.M, p.groups, tile_m);
    ntiles = static_cast<int32_t*>(ws);
    tiles = reinterpret_cast<Tile*>(static_cast<char*>(ws) + 256);
    fp8_tiles_kernel<<<1, 1024, 0, s>>>(offsets, p.groups, p.M, tile_m, max_tiles, tiles, ntiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return out_bf16 ? launch<uint16_t>(p, tiles, ntiles, max_tiles, stream, s)
                  : launch<float>(p, tiles, ntiles, max_tiles, stream, s);
}

}  // namespace lmoe
